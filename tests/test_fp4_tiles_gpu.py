"""GPU tests of the persistent fp4 product by its tiles: the pair of CTAs (256 channels x 192 rows) and the
single CTA's 128 rows, which the products of test_fp4_gpu hardly reach.  Every shape here says which tile it
is for, and a test that got another one fails, so that a change of the rule cannot take the tests away.
Compared as in test_fp4_gpu, with the tolerance derived there.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np
import pytest
import torch

import fp4_ref as ref
from rotated_w4a4_quantized_group_b200 import ck
from test_fp4_gpu import BF16, DT, F16, F32, FMT, MX, NV, _close, _gen, _t, _weights, _x, _xvalues

pytestmark = pytest.mark.gpu

PAIR, ONE = (2, 192), (1, 128)
# M, N, K of one matrix.  Channels end in the first and in the second CTA's half of the last tile; K ends in a
# stage and in a step of 64; one, two, three and eighteen tiles for the busiest pair; two to seventeen stages.
LINEARS = [(PAIR, 1500, 2049, 4112), (PAIR, 1400, 2178, 4128), (PAIR, 2400, 3840, 4096), (PAIR, 4097, 2178, 1040),
           (PAIR, 8000, 8000, 272), (ONE, 2500, 2050, 544), (ONE, 700, 2170, 1040)]
# the experts' offsets, N, K: rows before the first and behind the last, experts without rows, tiles that start
# anywhere in a 128-row block
EXPERTS = [(PAIR, (7, 700, 700, 1500, 2001), 1300, 4096), (PAIR, (0, 1193, 1200, 1999, 2001), 1410, 4112),
           (ONE, (3, 400, 401, 900, 1190), 1300, 4096)]


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
    _weights_of.cache_clear()
    torch.cuda.synchronize()


@functools.lru_cache(maxsize=2)
def _weights_of(E, N, K, fmt):
    return _weights(E, N, K, fmt, 100 + E, [0.0007 * (1 + e % 3) for e in range(E)] if fmt == NV else None)


def _wts(E, fmt):
    return None if fmt == MX else torch.tensor([0.0007 * (1 + e % 3) for e in range(E)], device="cuda")


# ------------------------------------------------------------------- one matrix

@FMT
@pytest.mark.parametrize("want,M,N,K", LINEARS)
def test_linear_of_a_tile(fmt, want, M, N, K):
    K = width(K, fmt)
    dt = (BF16, F16, F32)[(M + N + fmt) % 3]
    tx = 0.013 if fmt == NV else None
    x = _x(M, K, dt, 101, spread=False)
    w, ws, wv = _weights_of(1, N, K, fmt)
    bias = (torch.randn(N, generator=_gen(102)) * 0.3).to(dt).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xv = _xvalues(x, fmt, tx)
    exact, mag = xv @ wv[0].t() + bias.double(), xv.abs() @ wv[0].abs().t() + bias.double().abs()
    del xv
    kw = dict(x_tensor_scale=_t(tx), w_tensor_scale=_wts(1, fmt), dev_status=status)
    codes, scales = ck.ck_quant_fp4(x.cuda(), fmt, tensor_scale=_t(tx))
    for pad, first in ((-N % 8 + 8, 0), (3, 1)):        # 16-byte rows, and rows at any address
        assert tile(M, N, K, fmt, ragged=dt != F32 and (pad, first) == (3, 1)) == want
        buf = torch.full((M + 2, N + pad), 7.25, dtype=dt, device="cuda")
        out = buf[1:1 + M, first:first + N]
        ck.ck_fp4_linear(x.cuda(), w[0], ws[0], fmt, bias, out=out, **kw)
        _close(out, exact, mag, K, f"pad {pad}")
        assert torch.equal(out, ck.ck_fp4_linear(codes, w[0], ws[0], fmt, bias, x_scales=scales, out_dtype=dt, **kw))
        buf[1:1 + M, first:first + N] = 7.25
        assert (buf == 7.25).all()
    assert status.item() == 0


@FMT
@pytest.mark.parametrize("want,M,N,K", [(PAIR, 1500, 2178, 4096), (PAIR, 8000, 8000, 256), (ONE, 900, 2100, 768)])
def test_small_integers_are_exact(fmt, want, M, N, K):
    """Unit scales and codes: every partial sum is a multiple of 1/4 below 36 K, exact in fp32."""
    assert tile(M, N, K, fmt) == want
    g = np.random.default_rng(M)
    xc, wc = g.integers(0, 16, (M, K), dtype=np.uint8), g.integers(0, 16, (N, K), dtype=np.uint8)
    one, b = (127 if fmt == MX else 0x38), ref.BLOCK[fmt]
    xs = torch.from_numpy(ref.tile(np.full((M, K // b), one, np.uint8))).cuda()
    ws = torch.from_numpy(ref.tile(np.full((N, K // b), one, np.uint8))).cuda()
    out = ck.ck_fp4_linear(torch.from_numpy(ref.pack(xc)).cuda(), torch.from_numpy(ref.pack(wc)).cuda(), ws, fmt,
                           x_scales=xs, out_dtype=F32)
    exact = torch.from_numpy(ref.code_values(xc)).cuda() @ torch.from_numpy(ref.code_values(wc)).cuda().t()
    assert torch.equal(out.double(), exact)


@FMT
@pytest.mark.parametrize("want,M,N,K", [(PAIR, 1500, 2178, 4096), (ONE, 900, 2100, 768)])
def test_every_scale_reaches_its_own_block(fmt, want, M, N, K):
    """One nonzero element per row of x and power-of-two scales that differ for every row and block: each
    output is one product, exact in fp32."""
    assert tile(M, N, K, fmt) == want
    b, g = ref.BLOCK[fmt], np.random.default_rng(N)
    lo, hi = (120, 135) if fmt == MX else (1, 15)
    xe, we = g.integers(lo, hi, (M, K // b)), g.integers(lo, hi, (N, K // b))
    xb, wb = (xe if fmt == MX else xe << 3).astype(np.uint8), (we if fmt == MX else we << 3).astype(np.uint8)
    xc = np.zeros((M, K), np.uint8)
    xc[np.arange(M), g.integers(0, K, M)] = g.integers(1, 8, M)
    wc = g.integers(1, 16, (N, K), dtype=np.uint8)
    out = ck.ck_fp4_linear(torch.from_numpy(ref.pack(xc)).cuda(), torch.from_numpy(ref.pack(wc)).cuda(),
                           torch.from_numpy(ref.tile(wb)).cuda(), fmt, x_scales=torch.from_numpy(ref.tile(xb)).cuda(),
                           out_dtype=F32)
    exact = torch.from_numpy(ref.values(xc, xb, fmt)).cuda() @ torch.from_numpy(ref.values(wc, wb, fmt)).cuda().t()
    assert torch.equal(out.double(), exact)


@FMT
def test_nan_stays_in_its_row_and_channel_of_a_pair(fmt):
    M, N, K = 1400, 2178, 4128
    assert tile(M, N, K, fmt) == PAIR
    x = _x(M, K, BF16, 103, spread=False)
    rows, channels = [0, 95, 96, 191, 192, 1399], [0, 127, 128, 255, 256, 2177]
    for i, r in enumerate(rows):
        x[r, 700 * i] = float("nan") if i % 2 else float("inf")
    w, ws, wv = _weights_of(1, N, K, fmt)
    ws = ws.clone()
    at = ref.tile_index(channels, K // ref.BLOCK[fmt])
    for i in range(len(channels)):
        ws[0, at[i, 20 * i]] = 0xFF if fmt == MX else 0x7F
    out = ck.ck_fp4_linear(x.cuda(), w[0], ws[0], fmt, w_tensor_scale=_wts(1, fmt))
    want = torch.zeros(M, N, dtype=torch.bool)
    want[rows], want[:, channels] = True, True
    assert torch.equal(torch.isnan(out).cpu(), want)
    xv = _xvalues(x, fmt, None).nan_to_num(0.0)
    keep = ~want.cuda()
    _close(out[keep], (xv @ wv[0].t())[keep], (xv.abs() @ wv[0].abs().t())[keep], K)


@FMT
@pytest.mark.parametrize("M,N,K", [(1, 28677, 4096), (8, 40000, 1040), (16, 20001, 2064), (3, 151936, 272), (2, 30000, 16400)])
def test_few_rows_of_many_channels(fmt, M, N, K):
    """More tiles of 128 channels than run at once, the rows quantized in each.  The weights are quantized and
    read back by the library, bit for bit what the reference gives."""
    K = width(K, fmt)
    assert ck.fp4_workspace_bytes(M, K, fmt) == 0                # quantized inside
    g = torch.Generator(device="cuda").manual_seed(N)
    w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
    x = _x(M, K, F32, 106, spread=False)
    bias = torch.randn(N, device="cuda", generator=g)
    buf = torch.full((M + 2, N + 3), 7.25, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ck.ck_fp4_linear(x.cuda(), w, ws, fmt, bias, out=buf[1:1 + M, 1:1 + N], dev_status=status)
    assert status.item() == 0
    xv = _xvalues(x, fmt, None)
    for lo in range(0, N, 32768):                                # in 64 bits, some channels at a time
        n = slice(lo, min(lo + 32768, N))
        wv = ck.ck_dequant_fp4(w, ws, fmt, out_dtype=F32)[n].double()
        b = bias[n].double()
        _close(out[:, n], xv @ wv.t() + b, xv.abs() @ wv.abs().t() + b.abs(), K, f"channels from {lo}")
    buf[1:1 + M, 1:1 + N] = 7.25
    assert (buf == 7.25).all()


# ------------------------------------------------------------------- bytes of tiles that stand for no block

def _dirty(tiles, rows, blocks, fmt, seed):
    """Scale tiles with other bytes where no block is: behind the last block anything but a NaN, in rows behind
    the last anything."""
    g = np.random.default_rng(seed)
    any_byte, number = g.integers(0, 256, tiles.numel()), g.integers(0, 255, tiles.numel())
    if fmt == NV:
        number[number % 128 == 127] = 0x7E
    wide, last = -(-blocks // 4) * 4, -(-rows // 128) * 128
    out = any_byte.copy()
    at = ref.tile_index(np.arange(rows), wide)
    out[at] = number[at]
    at = at[:, :blocks]
    out[at] = tiles.cpu().numpy().reshape(-1)[at]
    assert wide > blocks and last > rows and out.size == last * wide
    return torch.from_numpy(out.astype(np.uint8)).view(tiles.shape).cuda()


@FMT
@pytest.mark.parametrize("want,M,N,steps", [(None, 5, 200, 1), (None, 9, 200, 6), ((0, 64), 40, 200, 6),
                                            ((0, 64), 100, 907, 16), ((1, 64), 400, 1600, 4), (ONE, 900, 2100, 3),
                                            (PAIR, 1500, 2178, 16)])
def test_padding_of_scale_tiles_does_not_matter(fmt, want, M, N, steps):
    """K ends one, two or three blocks into its last 64 (MX: one)."""
    b = ref.BLOCK[fmt]
    for K in (256 * steps + b * j for j in range(1, 64 // b)):
        assert want is None or tile(M, N, K, fmt) == want
        g = torch.Generator(device="cuda").manual_seed(K)
        x = torch.randn(M, K, device="cuda", generator=g, dtype=BF16)
        w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
        codes, xs = ck.ck_quant_fp4(x, fmt)
        ws2, xs2 = _dirty(ws, N, K // b, fmt, 1), _dirty(xs, M, K // b, fmt, 2)
        exact = ck.ck_fp4_linear(x, w, ws, fmt)
        assert torch.equal(exact, ck.ck_fp4_linear(x, w, ws2, fmt))
        assert torch.equal(exact, ck.ck_fp4_linear(codes, w, ws2, fmt, x_scales=xs2))
        assert torch.equal(ck.ck_dequant_fp4(codes, xs, fmt), ck.ck_dequant_fp4(codes, xs2, fmt))


# ------------------------------------------------------------------- by expert

@FMT
@pytest.mark.parametrize("want,off,N,K", EXPERTS)
def test_experts_of_a_tile(fmt, want, off, N, K):
    """Activations and codes in."""
    K, M, E = width(K, fmt), off[-1] + 9, len(off) - 1
    assert tile(M, N, K, fmt, E) == want
    dt = (BF16, F16, F32)[(N + fmt) % 3]
    tx = 0.02 if fmt == NV else None
    x = _x(M, K, dt, 104, spread=False)
    w, ws, wv = _weights_of(E, N, K, fmt)
    bias = (torch.randn(E, N, generator=_gen(105)) * 0.3).to(dt).cuda()
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = ck.ck_quant_fp4(x.cuda(), fmt, tensor_scale=_t(tx), offsets=offsets)
    xv = _xvalues(x, fmt, tx)
    for a, kw in ((x.cuda(), {}), (codes, dict(x_scales=scales))):
        out = torch.full((M, N + 6), -7.5, dtype=dt, device="cuda")
        ck.ck_fp4_expert_linear(a, offsets, w, ws, fmt, bias, x_tensor_scale=_t(tx), w_tensor_scale=_wts(E, fmt),
                                out=out[:, :N], dev_status=status, **kw)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            exact = xv[lo:hi] @ wv[e].t() + bias[e].double()
            mag = xv[lo:hi].abs() @ wv[e].abs().t() + bias[e].double().abs()
            _close(out[lo:hi, :N], exact, mag, K, f"expert {e}")
        assert (out[:off[0]] == -7.5).all() and (out[off[-1]:] == -7.5).all() and (out[:, N:] == -7.5).all()
    assert status.item() == 0


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


@FMT
@pytest.mark.parametrize("M", [3000, 2400])
def test_a_captured_pair_follows_its_inputs(fmt, M):
    N, K = 3840, 4096
    assert tile(M, N, K, fmt) == PAIR
    g = torch.Generator(device="cuda").manual_seed(120)
    x = torch.randn(M, K, device="cuda", generator=g, dtype=BF16)
    w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
    ck.ck_fp4_linear(x, w, ws, fmt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ck.ck_fp4_linear(x, w, ws, fmt)
    for _ in range(3):
        x.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ck.ck_fp4_linear(x, w, ws, fmt))


# ------------------------------------------------------------------- waits that run out

@FMT
@DT
@pytest.mark.parametrize("M,N,K,E", [(3000, 2048, 4096, 0), (2000, 1300, 4096, 4)])
def test_wait_expiry_of_a_pair(fmt, dt, M, N, K, E):
    """The build whose role waits give up at once: the call returns CK_OK, the status word says timeout, and
    a normal call afterwards gives what one before did."""
    assert tile(M, N, K, fmt, E) == PAIR
    L = ck.load_library(os.path.join(os.path.dirname(ck.LIB_PATH), "libck_test_waits.so"))
    g = torch.Generator(device="cuda").manual_seed(130)
    x = torch.randn(M, K, device="cuda", generator=g).to(dt)
    made = [ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt) for _ in range(max(E, 1))]
    w, ws = torch.stack([c for c, _ in made]), torch.stack([s for _, s in made])
    off = torch.tensor([0, 600, 600, 1500, 2000], dtype=torch.int32, device="cuda")

    def call(status):
        if E:
            return ck.ck_fp4_expert_linear(x, off, w, ws, fmt, dev_status=status)
        return ck.ck_fp4_linear(x, w[0], ws[0], fmt, dev_status=status)

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(status)
    out = torch.empty(M, N, dtype=dt, device="cuda")
    work = torch.empty(ck.fp4_workspace_bytes(M, K, fmt, E), dtype=torch.uint8, device="cuda")
    head = (x.data_ptr(), ck.DTYPE_CODE[dt], M, K, K, 1, fmt, None, None)
    tail = (ws.data_ptr(), None, None, 0, out.data_ptr(), ck.DTYPE_CODE[dt], N, work.data_ptr(), work.numel(),
            status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        status.zero_()
        if E:
            rc = L.ck_fp4_expert_linear(*head, off.data_ptr(), E, w.data_ptr(), N, K // 2, w.stride(0), *tail)
        else:
            rc = L.ck_fp4_linear(*head, w.data_ptr(), N, K // 2, *tail)
        assert rc == ck.CK_OK
        torch.cuda.synchronize()
        assert status.item() == ck.CK_ERR_TIMEOUT
        status.zero_()
        assert torch.equal(call(status), want)
        assert status.item() == 0
