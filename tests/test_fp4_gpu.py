"""GPU tests of the microscaled fp4 operators against float64.

Quantizing and reading back are compared bit for bit: the definition leaves no freedom.  Products
are compared bit for bit where every partial sum is exact in fp32, and otherwise within
    |got - exact| <= A * sum_k |x w| + half a step of the output type * |exact|
with A = (K / 16 + 8) * 2^-23: at most one addition per 16 products reaches the fp32 accumulator
(the products inside one are summed with more bits), each off by at most one step (2^-23 of the
running magnitude, which is at most sum |x w|) should the unit cut and not round; 8 covers the
products with the tensor scales and the bias' addition.
"""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch

import fp4_ref as ref
from rotated_w4a4_quantized_group_b200 import ck

pytestmark = pytest.mark.gpu

MX, NV = ck.CK_MXFP4, ck.CK_NVFP4
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FMT = pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
DT = pytest.mark.parametrize("dt", [BF16, F16, F32], ids=["bf16", "f16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.lib()
    yield
    torch.cuda.synchronize()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _x(M, K, dt, seed=0, spread=True):
    g = _gen(seed * 7919 + M * 31 + K)
    x = torch.randn(M, K, generator=g)
    if spread:   # blocks of very different size, zeros among them
        x *= torch.exp2(torch.randint(-6, 7, (M, 1), generator=g).float())
        x *= torch.where(torch.rand(1, K, generator=g) < 0.02, 20.0, 1.0)
        x[torch.rand(M, K, generator=g) < 0.05] = 0.0
    return x.to(dt)


def _place(x, layout):
    """x on the GPU in a layout: rows, a row pitch, an odd start, columns, every second element."""
    M, K = x.shape
    d = x.cuda()
    if layout == "rows":
        return d
    if layout == "pitch":
        buf = torch.full((M, K + 40), 7.0, dtype=x.dtype, device="cuda")
        buf[:, :K] = d
        return buf[:, :K]
    if layout == "odd":
        buf = torch.full((M, K + 3), 7.0, dtype=x.dtype, device="cuda")
        buf[:, 1: K + 1] = d
        return buf[:, 1: K + 1]
    if layout == "cols":
        return d.t().contiguous().t()
    if layout == "oddcols":
        buf = torch.full((K, M + 5), 7.0, dtype=x.dtype, device="cuda")
        buf[:, 1: M + 1] = d.t()
        return buf[:, 1: M + 1].t()
    buf = torch.full((M, 2 * K), 7.0, dtype=x.dtype, device="cuda")
    buf[:, ::2] = d
    return buf[:, ::2]


def _t(v):
    return None if v is None else torch.tensor([v], dtype=F32, device="cuda")


def _check_quant(x, fmt, t=None, layout="rows"):
    M, K = x.shape
    codes, scales = ck.ck_quant_fp4(_place(x, layout), fmt, tensor_scale=_t(t))
    torch.cuda.synchronize()
    rc, rs = ref.quantize(x, fmt, t)
    np.testing.assert_array_equal(scales.cpu().numpy(), ref.tile(rs))
    np.testing.assert_array_equal(ref.unpack(codes.cpu().numpy()), rc)
    return codes, scales, rc, rs


# ------------------------------------------------------------------- quantize

@FMT
@DT
@pytest.mark.parametrize("M,K", [(1, 32), (1, 3840), (3, 96), (17, 256), (127, 288), (128, 512),
                                 (129, 544), (300, 1056)])
def test_quant_bit_exact(fmt, dt, M, K):
    _check_quant(_x(M, K, dt), fmt)
    if fmt == NV:
        _check_quant(_x(M, K, dt, 1), fmt, t=0.0123)
        if K % 32 == 0 and K > 32:
            _check_quant(_x(M, K - 16, dt, 2), fmt)       # K ends inside a scale tile


@FMT
@DT
@pytest.mark.parametrize("layout", ["pitch", "odd", "cols", "oddcols", "second"])
@pytest.mark.parametrize("M,K", [(5, 64), (32, 96), (150, 352), (256, 320)])
def test_quant_layouts(fmt, dt, layout, M, K):
    _check_quant(_x(M, K, dt, 3), fmt, t=0.37 if fmt == NV else None, layout=layout)


@DT
@pytest.mark.parametrize("t", [None, 1.0, 0.3, 1.7e-3, 3.0] + [n / 2688 for n in (
    79, 84, 63, 128, 101.5, 147, 201, 0.33, 6.5625, 255, 171)])
def test_nv_borders(dt, t):
    """Values on and next to every border between two codes, for every E4M3 scale: x / (s t) on the
    border itself (rounded to x's type), one step below and one above."""
    t32 = np.float32(1.0 if t is None else t)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in ref.E4M3[1:]:
        d = np.float64(np.float32(np.float32(s) * t32))
        m = torch.from_numpy(mids * d).to(dt)
        near = [m, torch.nextafter(m, torch.full_like(m, 1e30)), torch.nextafter(m, torch.zeros_like(m))] \
            if dt == F32 else [m, (m.view(torch.int16) + 1).view(dt), (m.view(torch.int16) - 1).view(dt)]
        top = torch.tensor([6.0 * d]).to(dt)              # sets the block's scale to about s
        for v in near:
            rows.append(torch.cat([v, -v, top, torch.zeros(1, dtype=dt)]))
    _check_quant(torch.stack(rows), NV, t=t)


@DT
def test_nv_borders_of_short_tensor_scales(dt):
    """Tensor scales of few bits put whole sets of borders onto x's values: powers of two, and 1 / 2688 of a
    16-bit absmax in fp32 and rounded to that type."""
    g = _gen(5)
    m = (1 + torch.randint(0, 128, (14,), generator=g) / 128).tolist() + \
        (1 + torch.randint(0, 1024, (10,), generator=g) / 1024).tolist()
    ts = [2.0 ** -9, 2.0, 1.5, 1.25, 1.75]
    for i, a in enumerate(m):
        t = torch.tensor(a) / 2688
        ts += [t.item(), t.to(BF16 if i % 2 else F16).float().item(), a]
    for t in ts:
        test_nv_borders(dt, t)


@DT
def test_nv_scale_borders(dt):
    """Block maxima on and next to the borders between two E4M3 scales."""
    mid = torch.from_numpy((ref.E4M3[1:] + ref.E4M3[:-1]) / 2 * 6.0)
    for t in (None, 0.77):
        m = (mid * (1.0 if t is None else float(np.float32(t)))).to(dt)
        cand = [m]
        if dt == F32:
            cand += [torch.nextafter(m, torch.full_like(m, 1e30)), torch.nextafter(m, torch.zeros_like(m))]
        else:
            cand += [(m.view(torch.int16) + 1).view(dt), (m.view(torch.int16) - 1).view(dt)]
        x = torch.zeros(3 * len(m), 16, dtype=dt)
        x[:, 5] = torch.cat(cand)
        x[:, 9] = -x[:, 5] / 3
        _check_quant(x, NV, t=t)


@DT
def test_mx_powers_and_ties(dt):
    """Block maxima at powers of two and next to them, down to the smallest and up to the largest of
    the type, with elements on the borders."""
    info = torch.finfo(dt)
    lo = {BF16: -133, F16: -24, F32: -149}[dt]
    hi = {BF16: 127, F16: 15, F32: 127}[dt]
    rows = []
    for e in range(lo, hi + 1):
        for f in (1.0, 1.5, 1.9):
            top = np.float64(f) * 2.0 ** e
            if top > info.max:
                continue
            u = 2.0 ** max(e - 2, -127)
            v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.1, 0.49, 1.1, 7.9]) * u
            v = np.minimum(np.concatenate([v, -v, [top, -top]]), top)
            v = np.maximum(v, -top)
            rows.append(torch.from_numpy(np.concatenate([v, np.zeros(6)])).to(dt))
    _check_quant(torch.stack(rows), MX)


@FMT
@DT
def test_quant_non_finite(fmt, dt):
    """A NaN or an infinity makes its block's scale NaN and its codes zero, and no other block's."""
    x = _x(8, 256, dt, 5)
    x[1, 3] = float("nan")
    x[2, 100] = float("inf")
    x[3, 255] = -float("inf")
    x[4, :] = float("nan")
    x[5, 17], x[5, 18] = float("nan"), float("inf")
    codes, scales, rc, rs = _check_quant(x, fmt)
    assert (rs == (0xFF if fmt == MX else 0x7F)).sum() > 4


@pytest.mark.parametrize("t", [1e-38, 2.0 ** -149, 1e-30, 2.0 ** -70, 1e30, 3e38])
def test_nv_extreme_tensor_scales(t):
    x = _x(40, 128, F32, 6)
    for k in (1.0, 1e-30, 1e30):
        _check_quant(x * k, NV, t=t)


@pytest.mark.parametrize("t", [0.0, -1.0, float("nan"), float("inf"), -0.0])
def test_nv_bad_tensor_scale_makes_every_scale_nan(t):
    x = _x(5, 64, BF16, 7)
    codes, scales = ck.ck_quant_fp4(x.cuda(), NV, tensor_scale=_t(t))
    got = ref.untile(scales.cpu().numpy(), 5, 4)
    assert (got == 0x7F).all() and (codes.cpu() == 0).all()


@FMT
def test_quant_leaves_what_is_not_its_own(fmt):
    """Guard bytes beside the codes' rows and behind the scales; odd code addresses."""
    M, K = 37, 352
    x = _x(M, K, BF16, 8)
    rc, rs = ref.quantize(x, fmt)
    buf = torch.full((M + 2, K // 2 + 11), 0xA5, dtype=torch.uint8, device="cuda")
    n = ck.fp4_scales_bytes(M, K, fmt)
    sb = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    ck.ck_quant_fp4(x.cuda(), fmt, codes=buf[1: M + 1, 3: K // 2 + 3], scales=sb)
    got = buf.cpu().numpy()
    np.testing.assert_array_equal(got[1: M + 1, 3: K // 2 + 3], ref.pack(rc))
    got[1: M + 1, 3: K // 2 + 3] = 0xA5
    assert (got == 0xA5).all() and (sb[n:] == 0xA5).all()
    np.testing.assert_array_equal(sb[:n].cpu().numpy(), ref.tile(rs))


OFFSETS = {
    "even": [0, 40, 80, 120], "empty": [0, 0, 130, 130, 130, 300, 300], "one": [0, 1, 2, 3, 4],
    "tail": [5, 133, 134, 390], "wide": [0, 128, 256, 257, 513], "none": [0, 0, 0],
    "many": list(range(0, 70 * 3 + 1, 3)),
}


@FMT
@pytest.mark.parametrize("name", OFFSETS)
def test_quant_by_expert(fmt, name):
    off = OFFSETS[name]
    M, K = off[-1] + 9, 320
    E = len(off) - 1
    x = _x(M, K, BF16, 9)
    codes = torch.full((M, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ck.fp4_scales_bytes(M, K, fmt, E),), 0xA5, dtype=torch.uint8, device="cuda")
    ck.ck_quant_fp4(x.cuda(), fmt, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"),
                    codes=codes, scales=scales)
    rc, rs = ref.quantize(x, fmt)
    rows, idx = ref.expert_scale_index(off, K // ref.BLOCK[fmt])
    want = np.full((M, K // 2), 0xA5, np.uint8)
    want[rows] = ref.pack(rc)[rows]
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy()[idx], rs[rows])
    # back again: rows of no expert keep what the buffer held
    out = torch.full((M, K), -77.0, dtype=F32, device="cuda")
    ck.ck_dequant_fp4(codes, scales, fmt, out=out,
                      offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    exact = np.full((M, K), -77.0)
    exact[rows] = ref.values(rc, rs, fmt)[rows]
    np.testing.assert_array_equal(out.cpu().numpy().astype(np.float64), exact)


@FMT
def test_bad_offsets_stay_inside(fmt):
    """Offsets out of range and decreasing: clamped, or empty; nothing outside the tensors is touched
    (the guards stay), and experts whose range is sound are right."""
    M, K = 200, 128
    off = [-50, 30, 10, 150, 2 ** 31 - 1]
    x = _x(M, K, BF16, 10)
    E = len(off) - 1
    n = ck.fp4_scales_bytes(M, K, fmt, E)
    sb = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    buf = torch.full((M + 8, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    ck.ck_quant_fp4(x.cuda(), fmt, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"),
                    codes=buf[4: M + 4], scales=sb)
    torch.cuda.synchronize()
    assert (sb[n:] == 0xA5).all() and (buf[:4] == 0xA5).all() and (buf[M + 4:] == 0xA5).all()
    rc, _ = ref.quantize(x, fmt)
    np.testing.assert_array_equal(buf[4: M + 4].cpu().numpy(), ref.pack(rc))


# ------------------------------------------------------------------- read back

@FMT
@DT
def test_dequant_every_code_and_scale(fmt, dt):
    n = 256 if fmt == MX else 128
    b = ref.BLOCK[fmt]
    K = 4 * b
    byte = np.arange(n, dtype=np.uint8).reshape(-1, 4)
    code = np.tile(np.arange(16, dtype=np.uint8), (n // 4, K // 16))
    codes = torch.from_numpy(ref.pack(code)).cuda()
    scales = torch.from_numpy(ref.tile(byte)).cuda()
    for t in (None,) if fmt == MX else (None, 0.1, 3e-7, 1e30):
        out = ck.ck_dequant_fp4(codes, scales, fmt, tensor_scale=_t(t), out_dtype=dt)
        with np.errstate(all="ignore"):
            v = ref.values(code, byte, fmt).astype(np.float32)
            v = v * np.float32(1.0 if t is None else t)
        want = torch.from_numpy(v).to(dt)
        assert torch.equal(torch.nan_to_num(out.cpu(), nan=123.0, posinf=1e4, neginf=-1e4),
                           torch.nan_to_num(want, nan=123.0, posinf=1e4, neginf=-1e4))


@FMT
@DT
@pytest.mark.parametrize("M,K", [(1, 32), (130, 416), (257, 768)])
def test_dequant_pitches_and_guards(fmt, dt, M, K):
    x = _x(M, K, F32, 11)
    rc, rs = ref.quantize(x, fmt)
    cb = torch.zeros(M, K // 2 + 5, dtype=torch.uint8, device="cuda")
    cb[:, 1: K // 2 + 1] = torch.from_numpy(ref.pack(rc)).cuda()
    ob = torch.full((M, K + 3), 5.5, dtype=dt, device="cuda")
    ck.ck_dequant_fp4(cb[:, 1: K // 2 + 1], torch.from_numpy(ref.tile(rs)).cuda(), fmt, out=ob[:, :K])
    want = torch.from_numpy(ref.values(rc, rs, fmt).astype(np.float32)).to(dt)
    assert torch.equal(ob[:, :K].cpu(), want) and (ob[:, K:] == 5.5).all()


# ------------------------------------------------------------------- products

def _weights(E, N, K, fmt, seed, t=None):
    """Quantized weights of E experts on the GPU, at a pitch of 16 bytes, and their values (E, N, K)
    in float64 (with the tensor scales)."""
    g = _gen(seed)
    pitch = -(-(K // 2) // 16) * 16
    buf = torch.full((E, N, pitch), 0x77, dtype=torch.uint8)
    sc, val = [], []
    for e in range(E):
        w = torch.randn(N, K, generator=g) * 0.05
        rc, rs = ref.quantize(w, fmt, None if t is None else t[e])
        buf[e, :, : K // 2] = torch.from_numpy(ref.pack(rc))
        sc.append(torch.from_numpy(ref.tile(rs)))
        v = torch.from_numpy(ref.values(rc, rs, fmt))
        val.append(v if t is None else v * float(np.float32(t[e])))
    return buf.cuda()[:, :, : K // 2], torch.stack(sc).cuda(), torch.stack(val).cuda()


def _xvalues(x, fmt, t):
    rc, rs = ref.quantize(x, fmt, t)
    v = torch.from_numpy(ref.values(rc, rs, fmt)).cuda()
    return v if t is None else v * float(np.float32(t))


def _close(got, exact, mag, K, what=""):
    dt = got.dtype
    tol = (K / 16 + 8) * 2.0 ** -23 * mag + torch.finfo(dt).eps / 2 * exact.abs() * (1 + 2.0 ** -8)
    if dt == F16:
        tol = tol + 2.0 ** -25        # half a step of its subnormals
    err = (got.double() - exact).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: off by {worst:.3g} more than the bound"


SHAPES = [(1, 1, 32), (3, 5, 16), (70, 9, 16), (1, 3840, 3840), (7, 200, 16384), (8, 96, 272), (9, 4000, 1040), (15, 333, 10240), (16, 129, 16400),
          (17, 130, 12320), (40, 200, 12304), (1, 300, 46080), (2, 260, 23040), (16, 150, 2816), (64, 300, 40000), (2, 40, 64), (5, 300, 96), (16, 130, 800), (31, 257, 1056),
          (33, 640, 2080), (64, 128, 256), (65, 129, 288), (100, 1111, 2064), (127, 500, 512),
          (128, 256, 4096), (200, 384, 1024), (413, 1111, 2064), (700, 1920, 544), (1500, 2049, 1040),
          (2500, 3840, 320), (4097, 1300, 272)]


@FMT
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(fmt, M, N, K):
    if K % ref.BLOCK[fmt]:
        K += 16
    dt = (BF16, F16, F32)[(M + N) % 3]
    tx, tw = (0.013, [0.0007]) if fmt == NV and M % 2 else (None, None)
    x = _x(M, K, dt, 12, spread=False)
    w, ws, wv = _weights(1, N, K, fmt, 13, tw)
    bias = (torch.randn(N, generator=_gen(14)) * 0.3).to(dt).cuda() if N % 2 else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ck.ck_fp4_linear(x.cuda(), w[0], ws[0], fmt, bias, x_tensor_scale=_t(tx),
                           w_tensor_scale=_t(tw[0]) if tw else None, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and out.dtype == dt
    xv = _xvalues(x, fmt, tx)
    exact, mag = xv @ wv[0].t(), xv.abs() @ wv[0].abs().t()
    if bias is not None:
        exact, mag = exact + bias.double(), mag + bias.double().abs()
    _close(out, exact, mag, K)


@FMT
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(65, 64, 3840), (100, 907, 10240), (128, 640, 2048), (191, 130, 16640),
                                   (257, 300, 46080), (300, 1111, 4128), (640, 388, 2848), (1000, 60, 5120)])
def test_linear_of_few_tiles(fmt, dt, M, N, K):
    """K split over several CTAs a tile, with tiles of rows that end inside a tile of scales: activations
    and codes in, an output with a pitch, and the rows and columns around it left alone."""
    x = _x(M, K, dt, 15, spread=False)
    w, ws, wv = _weights(1, N, K, fmt, 16)
    bias = (torch.randn(N, generator=_gen(17)) * 0.3).to(dt).cuda()
    codes, scales = ck.ck_quant_fp4(x.cuda(), fmt)
    xv = _xvalues(x, fmt, None)
    exact, mag = xv @ wv[0].t() + bias.double(), xv.abs() @ wv[0].abs().t() + bias.double().abs()
    for pad, first in ((8, 0), (5, 1)):
        buf = torch.full((M + 2, N + pad), 7.25, dtype=dt, device="cuda")
        out = buf[1:1 + M, first:first + N]
        ck.ck_fp4_linear(codes, w[0], ws[0], fmt, bias, x_scales=scales, out=out)
        _close(out, exact, mag, K, f"pad {pad}")
        buf[1:1 + M, first:first + N] = 7.25
        assert (buf == 7.25).all()
    buf = torch.empty(M, N, dtype=dt, device="cuda")
    again = ck.ck_fp4_linear(x.cuda(), w[0], ws[0], fmt, bias, out=buf)
    assert torch.equal(again, ck.ck_fp4_linear(x.cuda(), w[0], ws[0], fmt, bias))
    _close(again, exact, mag, K, "activations")


@FMT
@pytest.mark.parametrize("M,N,K", [(7, 130, 512), (70, 300, 1024), (300, 900, 768), (3000, 2000, 512)])
def test_product_of_small_integers_is_exact(fmt, M, N, K):
    """Unit scales and codes: every partial sum is a multiple of 1/4 below 36 K, exact in fp32."""
    g = np.random.default_rng(M)
    xc = g.integers(0, 16, (M, K), dtype=np.uint8)
    wc = g.integers(0, 16, (N, K), dtype=np.uint8)
    one = 127 if fmt == MX else 0x38
    b = ref.BLOCK[fmt]
    xs = torch.from_numpy(ref.tile(np.full((M, K // b), one, np.uint8))).cuda()
    ws = torch.from_numpy(ref.tile(np.full((N, K // b), one, np.uint8))).cuda()
    out = ck.ck_fp4_linear(torch.from_numpy(ref.pack(xc)).cuda(), torch.from_numpy(ref.pack(wc)).cuda(),
                           ws, fmt, x_scales=xs, out_dtype=F32)
    exact = torch.from_numpy(ref.code_values(xc)).cuda() @ torch.from_numpy(ref.code_values(wc)).cuda().t()
    assert torch.equal(out.double(), exact)


@FMT
@pytest.mark.parametrize("M,N,K", [(20, 260, 512), (400, 700, 1024)])
def test_every_scale_reaches_its_own_block(fmt, M, N, K):
    """One nonzero element per row of x and power-of-two scales that differ for every row and block:
    each output is one product, exact in fp32."""
    b = ref.BLOCK[fmt]
    g = np.random.default_rng(N)
    lo, hi = (120, 135) if fmt == MX else (1, 15)
    exps = g.integers(lo, hi, (M, K // b))
    wexps = g.integers(lo, hi, (N, K // b))
    xb = (exps if fmt == MX else exps << 3).astype(np.uint8)
    wb = (wexps if fmt == MX else wexps << 3).astype(np.uint8)
    xc = np.zeros((M, K), np.uint8)
    at = g.integers(0, K, M)
    xc[np.arange(M), at] = g.integers(1, 8, M)
    wc = g.integers(1, 16, (N, K), dtype=np.uint8)
    out = ck.ck_fp4_linear(torch.from_numpy(ref.pack(xc)).cuda(), torch.from_numpy(ref.pack(wc)).cuda(),
                           torch.from_numpy(ref.tile(wb)).cuda(), fmt,
                           x_scales=torch.from_numpy(ref.tile(xb)).cuda(), out_dtype=F32)
    exact = torch.from_numpy(ref.values(xc, xb, fmt)).cuda() @ \
        torch.from_numpy(ref.values(wc, wb, fmt)).cuda().t()
    assert torch.equal(out.double(), exact)


EXPERTS = [("even", 130, 256), ("empty", 300, 544), ("one", 128, 3840), ("tail", 257, 320),
           ("wide", 1111, 512), ("none", 64, 64), ("many", 140, 288)]


@FMT
@pytest.mark.parametrize("name,N,K", EXPERTS)
def test_expert_linear(fmt, name, N, K):
    off = OFFSETS[name]
    M, E = off[-1] + 9, len(off) - 1
    dt = (BF16, F16, F32)[N % 3]
    tw = [0.001 * (1 + e % 5) for e in range(E)] if fmt == NV else None
    tx = 0.02 if fmt == NV else None
    x = _x(M, K, dt, 15, spread=False)
    w, ws, wv = _weights(E, N, K, fmt, 16, tw)
    bias = (torch.randn(E, N, generator=_gen(17)) * 0.3).to(F32).cuda() if N % 2 else None
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    out = torch.full((M, N + 8), -7.5, dtype=dt, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ck.ck_fp4_expert_linear(x.cuda(), offsets, w, ws, fmt, bias, x_tensor_scale=_t(tx),
                            w_tensor_scale=None if tw is None else torch.tensor(tw, device="cuda"),
                            out=out[:, :N], dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
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


# ------------------------------------------------------------------- values that are not numbers

@FMT
@pytest.mark.parametrize("M,N", [(6, 200), (40, 200), (300, 1000)])
def test_nan_stays_in_its_row_and_channel(fmt, M, N):
    """A NaN activation makes its row's outputs NaN, a weight block with a NaN scale its channel's,
    and nothing else."""
    K = 320
    x = _x(M, K, BF16, 20, spread=False)
    x[2, 70] = float("nan")
    x[5, 300] = float("inf")
    w, ws, wv = _weights(1, N, K, fmt, 21)
    n = N - 60
    ws[0, ref.tile_index([n], K // ref.BLOCK[fmt])[0, 3]] = 0xFF if fmt == MX else 0x7F
    out = ck.ck_fp4_linear(x.cuda(), w[0], ws[0], fmt)
    bad = torch.isnan(out).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[2], want[5], want[:, n] = True, True, True
    assert torch.equal(bad, want)
    xv = _xvalues(x, fmt, None).nan_to_num(0.0)
    exact, mag = xv @ wv[0].t(), xv.abs() @ wv[0].abs().t()
    keep = ~want.cuda()
    _close(out[keep], exact[keep], mag[keep], K)


def test_fp16_output_overflows_to_infinity():
    x = torch.full((40, 64), 6.0, dtype=F16)
    w = torch.from_numpy(ref.pack(np.full((8, 64), 7, np.uint8))).cuda()
    ws = torch.from_numpy(ref.tile(np.full((8, 2), 140, np.uint8))).cuda()      # 2^13
    out = ck.ck_fp4_linear(x.cuda(), w, ws, MX)
    assert torch.isinf(out).all() and (out > 0).all()


# ------------------------------------------------------------------- how calls are made

def _case(fmt, M, N, K, dt=BF16, seed=30):
    x = _x(M, K, dt, seed, spread=False).cuda()
    w, ws, _ = _weights(1, N, K, fmt, seed + 1)
    return x, w[0], ws[0]


@FMT
@pytest.mark.parametrize("M", [3, 40, 500])
def test_same_bits_every_time(fmt, M):
    x, w, ws = _case(fmt, M, 700, 1056)
    first = ck.ck_fp4_linear(x, w, ws, fmt)
    for _ in range(5):
        assert torch.equal(first, ck.ck_fp4_linear(x, w, ws, fmt))


@FMT
@pytest.mark.parametrize("M", [1, 17, 64, 65, 300])
def test_codes_in_equal_activations_in(fmt, M):
    """ck_quant_fp4 and then the product of codes gives the bits of the product of activations, also
    where that quantizes inside its own kernel."""
    x, w, ws = _case(fmt, M, 333, 1056)
    t = _t(0.031) if fmt == NV else None
    codes, scales = ck.ck_quant_fp4(x, fmt, tensor_scale=t)
    a = ck.ck_fp4_linear(x, w, ws, fmt, x_tensor_scale=t)
    b = ck.ck_fp4_linear(codes, w, ws, fmt, x_scales=scales, x_tensor_scale=t)
    assert a.dtype == b.dtype == BF16 and torch.equal(a, b)


@FMT
@pytest.mark.parametrize("layout", ["pitch", "odd", "cols", "second"])
@pytest.mark.parametrize("M", [5, 40])
def test_linear_of_any_layout(fmt, layout, M):
    x, w, ws = _case(fmt, M, 130, 544)
    assert torch.equal(ck.ck_fp4_linear(x, w, ws, fmt),
                       ck.ck_fp4_linear(_place(x.cpu(), layout), w, ws, fmt))


@FMT
@pytest.mark.parametrize("M", [9, 40, 200])
def test_output_pitch_and_guards(fmt, M):
    N = 130
    x, w, ws = _case(fmt, M, N, 288)
    ref_out = ck.ck_fp4_linear(x, w, ws, fmt)
    for pad, first in ((6, 0), (8, 8), (7, 3)):
        buf = torch.full((M + 2, N + pad + first), -7.5, dtype=BF16, device="cuda")
        ck.ck_fp4_linear(x, w, ws, fmt, out=buf[1: M + 1, first: N + first])
        assert torch.equal(buf[1: M + 1, first: N + first], ref_out)
        buf[1: M + 1, first: N + first] = -7.5
        assert (buf == -7.5).all()


@FMT
@pytest.mark.parametrize("M", [4, 50, 300])
def test_captured_and_replayed_on_new_inputs(fmt, M):
    """A captured call follows its buffers; two graphs captured one after the other do not disturb each
    other."""
    x, w, ws = _case(fmt, M, 400, 544)
    y = x.clone()
    ck.ck_fp4_linear(x, w, ws, fmt)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = ck.ck_fp4_linear(x, w, ws, fmt)
    with torch.cuda.graph(g2):
        c2, s2 = ck.ck_quant_fp4(y, fmt)
        o2 = ck.ck_fp4_linear(c2, w, ws, fmt, x_scales=s2)
    for k in range(3):
        x.copy_(_x(M, 544, BF16, 40 + k, spread=False))
        y.copy_(_x(M, 544, BF16, 50 + k, spread=False))
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, ck.ck_fp4_linear(x, w, ws, fmt))
        assert torch.equal(o2, ck.ck_fp4_linear(y, w, ws, fmt))


@FMT
def test_captured_expert_call_follows_its_offsets(fmt):
    M, N, K, E = 300, 260, 288, 5
    x = _x(M, K, BF16, 60, spread=False).cuda()
    w, ws, _ = _weights(E, N, K, fmt, 61)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, dtype=BF16, device="cuda")
    ck.ck_fp4_expert_linear(x, off, w, ws, fmt, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ck_fp4_expert_linear(x, off, w, ws, fmt, out=out)
    for o in ([0, 100, 100, 200, 290, 300], [0, 0, 0, 0, 0, 300], [7, 8, 9, 10, 11, 12], [0] * 6):
        off.copy_(torch.tensor(o, dtype=torch.int32))
        out.fill_(-7.5)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        for e in range(E):
            if o[e + 1] > o[e]:
                one = ck.ck_fp4_linear(x[o[e]:o[e + 1]], w[e], ws[e], fmt)
                # the same codes and products; the sums' order may differ between the kernels
                assert torch.allclose(got[o[e]:o[e + 1]].float(), one.float(), rtol=2 ** -7, atol=1e-3)
        assert (got[:o[0]] == -7.5).all() and (got[o[-1]:] == -7.5).all()


@FMT
def test_one_row_and_one_channel_at_any_pitch(fmt):
    """A single row of codes, or a single channel's weights, needs no 16-byte pitch."""
    K = 96                                                       # 48 bytes a row
    x, w, ws = _case(fmt, 5, 1, K)
    want = ck.ck_fp4_linear(x, w, ws, fmt)
    tight = w.contiguous().clone()
    assert torch.equal(ck.ck_fp4_linear(x, tight, ws, fmt), want)
    codes, scales = ck.ck_quant_fp4(x[:1], fmt)
    for c in (codes, codes.contiguous().clone(), codes.expand(1, K // 2).clone()):
        assert torch.equal(ck.ck_fp4_linear(c, tight, ws, fmt, x_scales=scales), want[:1])


@FMT
def test_as_many_experts_as_a_call_takes(fmt):
    E, N, K = 1024, 40, 64
    g = torch.Generator().manual_seed(8)
    count = torch.randint(0, 4, (E,), generator=g)
    off = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    M = int(off[-1])
    x = _x(M, K, BF16, 31, spread=False)
    wc = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    byte = np.random.default_rng(9).integers(*((120, 130) if fmt == MX else (40, 80)),
                                             (E, N, K // ref.BLOCK[fmt])).astype(np.uint8)
    ws = torch.from_numpy(np.stack([ref.tile(b) for b in byte])).cuda()
    out = ck.ck_fp4_expert_linear(x.cuda(), off.cuda(), wc.cuda(), ws, fmt)
    xv = _xvalues(x, fmt, None)
    wv = torch.from_numpy(ref.values(ref.unpack(wc.numpy()), byte, fmt)).cuda()
    w_of = wv[torch.repeat_interleave(torch.arange(E), count).cuda()]
    exact, mag = (xv[:, None] * w_of).sum(-1), (xv[:, None] * w_of).abs().sum(-1)
    _close(out, exact, mag, K)
    with pytest.raises(ck.CkError):
        two = torch.cat([off, off[-1:]]).cuda()
        ck.ck_fp4_expert_linear(x.cuda(), two, torch.cat([wc, wc[:1]]).cuda(), torch.cat([ws, ws[:1]]), fmt)


@FMT
def test_the_default_stream_by_its_handle(fmt):
    x, w, ws = _case(fmt, 40, 64, 128)
    want = ck.ck_fp4_linear(x, w, ws, fmt)
    torch.cuda.synchronize()
    for s in (0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream):
        codes, scales = ck.ck_quant_fp4(x, fmt, stream=s)
        got = ck.ck_fp4_linear(codes, w, ws, fmt, x_scales=scales, stream=s)
        ck.ck_dequant_fp4(codes, scales, fmt, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@FMT
@pytest.mark.parametrize("M", [12, 48, 400])
def test_two_calls_at_once_on_two_streams(fmt, M):
    x, w, ws = _case(fmt, M, 1000, 2080)
    y = _x(M, 2080, BF16, 70, spread=False).cuda()
    want = ck.ck_fp4_linear(x, w, ws, fmt), ck.ck_fp4_linear(y, w, ws, fmt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(6):
        got[0].append(ck.ck_fp4_linear(x, w, ws, fmt, stream=s[0]))
        got[1].append(ck.ck_fp4_linear(y, w, ws, fmt, stream=s[1].cuda_stream))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(o, b) for o in a)


def test_many_calls_at_once():
    """Calls on eight streams, pairs, clusters and single CTAs among them, more than the GPU holds at a
    time: none waits for tensor memory that a call waiting for it holds."""
    cases = [_case(NV if i % 2 else MX, M, N, K, seed=60 + i) + (NV if i % 2 else MX,)
             for i, (M, N, K) in enumerate([(2, 3840, 512), (8, 3840, 1024), (40, 3840, 2048), (100, 907, 4096),
                                            (600, 2048, 512), (1, 7680, 768), (33, 2048, 2816), (12, 3840, 2304)])]
    want = [ck.ck_fp4_linear(x, w, ws, fmt) for x, w, ws, fmt in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(40):
        for i, (x, w, ws, fmt) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(ck.ck_fp4_linear(x, w, ws, fmt))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(o, want[i]) for o in outs), f"case {i}"


@FMT
@DT
@pytest.mark.parametrize("M", [7, 40])
def test_broadcast_and_overlapping_activations(fmt, dt, M):
    _, w, ws = _case(fmt, 1, 130, 544)
    row, col = _x(1, 544, dt, 65).cuda(), _x(M, 1, dt, 66).cuda()
    flat = _x(1, 544 + 3 * M, dt, 67).cuda()[0]
    for x in (row.expand(M, 544), col.expand(M, 544), flat.as_strided((M, 544), (1, 1)),
              flat.as_strided((M, 544), (3, 1))):
        for a, b in zip(ck.ck_quant_fp4(x, fmt), ck.ck_quant_fp4(x.contiguous(), fmt)):
            assert torch.equal(a, b)
        assert torch.equal(ck.ck_fp4_linear(x, w, ws, fmt), ck.ck_fp4_linear(x.contiguous(), w, ws, fmt))


def test_what_a_call_would_write_past_is_refused():
    x, w, ws = _case(NV, 40, 64, 512)
    for kw in ({"dev_status": torch.zeros(4, dtype=torch.uint8, device="cuda")},
               {"dev_status": torch.zeros(0, dtype=torch.int32, device="cuda")},
               {"workspace": torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20)}):
        with pytest.raises(ValueError):
            ck.ck_fp4_linear(x, w, ws, NV, **kw)
    for fmt in (2, -1, 2 ** 70, None, "NV"):
        with pytest.raises(ValueError):
            ck.ck_fp4_linear(x, w, ws, fmt)


def test_callers_workspace_and_its_layout():
    M, N, K = 100, 200, 544
    x, w, ws = _case(NV, M, N, K)
    need = ck.fp4_workspace_bytes(M, K, NV)
    buf = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    out = ck.ck_fp4_linear(x, w, ws, NV, workspace=buf)
    assert torch.equal(out, ck.ck_fp4_linear(x, w, ws, NV)) and (buf[need:] == 0x5A).all()
    codes, scales = ck.ck_quant_fp4(x, NV)
    pitch = -(-K // 2 // 16) * 16
    at = -(-M * pitch // 256) * 256
    assert torch.equal(buf[: M * pitch].view(M, pitch)[:, : K // 2], codes)
    assert torch.equal(buf[at: at + scales.numel()], scales)
    with pytest.raises(ck.CkError):
        ck.ck_fp4_linear(x, w, ws, NV, workspace=buf[: need - 256])


def test_binding_refuses_what_does_not_fit():
    x, w, ws = _case(NV, 20, 64, 128)
    wt, off = _t(0.1), torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    w2, ws2, _ = _weights(2, 64, 128, NV, 80)
    bad = [lambda: ck.ck_fp4_linear(x, w[:, :60], ws, NV), lambda: ck.ck_fp4_linear(x, w, ws[:100], NV),
           lambda: ck.ck_fp4_linear(x, w, ws, NV, torch.zeros(63, device="cuda")),
           lambda: ck.ck_fp4_linear(x, w, ws, NV, out=torch.empty(20, 63, device="cuda")),
           lambda: ck.ck_fp4_linear(x, w, ws, MX, x_tensor_scale=wt),
           lambda: ck.ck_fp4_linear(x, w, ws, NV, w_tensor_scale=wt.double()),
           lambda: ck.ck_fp4_linear(x, w, ws, NV, w_tensor_scale=torch.ones(2, device="cuda")),
           lambda: ck.ck_fp4_linear(x.byte()[:, :64], w, ws, NV),
           lambda: ck.ck_fp4_linear(x, w.cpu(), ws, NV), lambda: ck.ck_fp4_linear(x, w.t(), ws, NV),
           lambda: ck.ck_fp4_expert_linear(x, off[:2], w2, ws2, NV),
           lambda: ck.ck_fp4_expert_linear(x, off.long(), w2, ws2, NV),
           lambda: ck.ck_fp4_expert_linear(x, off, w2, ws2[:, :-512], NV),
           lambda: ck.ck_fp4_expert_linear(x, off, w2, ws2, NV, torch.zeros(64, device="cuda")),
           lambda: ck.ck_quant_fp4(x, NV, tensor_scale=torch.ones(2, device="cuda")),
           lambda: ck.ck_quant_fp4(x, NV, codes=torch.empty(20, 63, dtype=torch.uint8, device="cuda")),
           lambda: ck.ck_quant_fp4(x, NV, scales=torch.empty(10, dtype=torch.uint8, device="cuda")),
           lambda: ck.ck_dequant_fp4(w, ws[:64], NV), lambda: ck.ck_dequant_fp4(w.char(), ws, NV)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    # weights at a pitch that TMA cannot read are refused by the library
    odd = torch.zeros(64, 72, dtype=torch.uint8, device="cuda")[:, :64]
    with pytest.raises(ck.CkError):
        ck.ck_fp4_linear(x, odd, ws, NV)


def test_past_two_to_the_31():
    """Rows whose element offsets need more than 32 bits: the last rows are right, in and out."""
    M, K, N = 140000, 16384, 16400
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(M, K, dtype=BF16, device="cuda").normal_(generator=g)
    codes, scales = ck.ck_quant_fp4(x, NV)
    y = ck.ck_dequant_fp4(codes, scales, NV)
    last = x[-3:].cpu()
    rc, rs = ref.quantize(last, NV)
    np.testing.assert_array_equal(ref.unpack(codes[-3:].cpu().numpy()), rc)
    np.testing.assert_array_equal(y[-3:].float().cpu().numpy().astype(np.float64), ref.values(rc, rs, NV))
    del y, codes, scales
    w, ws, wv = _weights(1, N, 64, NV, 6)
    out = ck.ck_fp4_linear(x[:, :64], w[0], ws[0], NV)
    xv = _xvalues(x[-3:, :64].cpu(), NV, None)
    _close(out[-3:], xv @ wv[0].t(), xv.abs() @ wv[0].abs().t(), 64)


# ------------------------------------------------------------------- together

@FMT
def test_a_mixture_of_experts_layer(fmt):
    """Router, sort, up projection, activation, down projection, weighted sum back: the operators as a
    layer uses them, its weights quantized by them too.  Each step is compared on the inputs that it
    got, so that no rounding of one step hides in another's tolerance."""
    T, D, H, E, top = 90, 320, 544, 6, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    tok = torch.randn(T, D, device="cuda", generator=g, dtype=BF16)
    up = torch.randn(E, H, D, device="cuda", generator=g) * 0.06
    down = torch.randn(E, D, H, device="cuda", generator=g) * 0.06

    def quantized(w):
        t = w.abs().amax((1, 2)) / (6 * 448) if fmt == NV else None
        both = [ck.ck_quant_fp4(w[e], fmt, tensor_scale=None if t is None else t[e: e + 1])
                for e in range(E)]
        # contiguous rows of 16-byte multiples, as the widths here are
        return torch.stack([c for c, _ in both]), torch.stack([s for _, s in both]), t

    def values(q):
        c, s, t = (v if v is None else v.cpu().numpy() for v in q)
        k = 2 * c.shape[-1] // ref.BLOCK[fmt]
        v = np.stack([ref.values(ref.unpack(c[e]), ref.untile(s[e], c.shape[1], k), fmt) for e in range(E)])
        return torch.from_numpy(v if t is None else v * t.astype(np.float64)[:, None, None]).cuda()

    qu, qd = quantized(up), quantized(down)
    prob, pick = torch.randn(T, E, device="cuda", generator=g).softmax(-1).topk(top)
    order = pick.flatten().argsort(stable=True)
    rows = order // top
    count = torch.bincount(pick.flatten(), minlength=E)
    off = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()

    def expert(x, q, out_dtype):
        out = ck.ck_fp4_expert_linear(x, off, q[0], q[1], fmt, w_tensor_scale=q[2], out_dtype=out_dtype)
        v, xv, o = values(q), _xvalues(x.cpu(), fmt, None), off.tolist()
        for e in range(E):
            a = xv[o[e]: o[e + 1]]
            _close(out[o[e]: o[e + 1]], a @ v[e].t(), a.abs() @ v[e].abs().t(), x.shape[1], f"expert {e}")
        return out

    h = expert(tok[rows], qu, BF16)
    h = torch.nn.functional.silu(h.float()).to(BF16)
    z = expert(h, qd, F32)
    y = torch.zeros(T, D, device="cuda").index_add_(0, rows, z * prob.flatten()[order][:, None])
    # The whole layer against the unquantized one.  E2M1's half step is at most a quarter of the value,
    # about 0.25 / sqrt(3) of it in the mean (0.14); four operands in two products, independent: 0.29.
    full = torch.zeros(T, D, device="cuda", dtype=torch.float64)
    for i in range(T):
        for j in range(top):
            e = int(pick[i, j])
            a = torch.nn.functional.silu(tok[i].double() @ up[e].double().t())
            full[i] += prob[i, j].double() * (a @ down[e].double().t())
    assert (y.double() - full).norm() < 0.35 * full.norm()


# ------------------------------------------------------------------- waits that run out

@FMT
@pytest.mark.parametrize("what,M,N,K,E", [("few rows, from activations", 8, 512, 1024, 0),
                                          ("few rows, from codes", 40, 512, 1024, 0),
                                          ("few rows, many steps", 40, 512, 30720, 0),
                                          ("one CTA a tile", 200, 256, 1024, 0),
                                          ("two CTAs a tile", 3000, 2048, 1024, 0),
                                          ("by expert", 300, 512, 1024, 4)])
def test_wait_expiry_returns_a_status(fmt, what, M, N, K, E):
    """The build whose role waits give up at once: the call returns CK_OK, the status word says timeout,
    and a normal call afterwards is right."""
    L = ck.load_library(os.path.join(os.path.dirname(ck.LIB_PATH), "libck_test_waits.so"))
    x = _x(M, K, BF16, 90, spread=False).cuda()
    w, ws, wv = _weights(max(E, 1), N, K, fmt, 91)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, dtype=BF16, device="cuda")
    work = torch.empty(max(ck.fp4_workspace_bytes(M, K, fmt, E), 256), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    head = (x.data_ptr(), ck.CK_BF16, M, K, K, 1, fmt, None, None)
    tail = (ws.data_ptr(), None, None, 0, out.data_ptr(), ck.CK_BF16, N, work.data_ptr(), work.numel(),
            status.data_ptr(), st)
    if E:
        off = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device="cuda")
        rc = L.ck_fp4_expert_linear(*head, off.data_ptr(), E, w.data_ptr(), N, K // 2, w.stride(0), *tail)
    else:
        rc = L.ck_fp4_linear(*head, w.data_ptr(), N, K // 2, *tail)
    assert rc == ck.CK_OK
    torch.cuda.synchronize()
    assert status.item() == ck.CK_ERR_TIMEOUT, what
    status.zero_()
    if not E:
        good = ck.ck_fp4_linear(x, w[0], ws[0], fmt, dev_status=status)
        xv = _xvalues(x.cpu(), fmt, None)
        _close(good, xv @ wv[0].t(), xv.abs() @ wv[0].abs().t(), K, what)
    else:
        good = ck.ck_fp4_expert_linear(x, off, w, ws, fmt, dev_status=status)
        xv = _xvalues(x[:100].cpu(), fmt, None)
        _close(good[:100], xv @ wv[0].t(), xv.abs() @ wv[0].abs().t(), K, what)
    assert status.item() == 0


# ------------------------------------------------------------------- both host sides

def _forms():
    """Call forms, sound ones and ones that are refused."""
    x, w, ws = _case(NV, 40, 200, 544)
    w3, ws3, _ = _weights(3, 64, 544, NV, 95)
    t, tw3 = _t(0.07), torch.tensor([0.1, 0.2, 0.3], device="cuda")
    off = torch.tensor([0, 10, 10, 35], dtype=torch.int32, device="cuda")
    codes, scales = ck.ck_quant_fp4(x, NV)
    ecodes, escales = ck.ck_quant_fp4(x, NV, offsets=off)
    bias, bias3 = torch.randn(200, device="cuda"), torch.randn(3, 64, device="cuda").half()
    work = torch.empty(ck.fp4_workspace_bytes(40, 544, NV), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L, X, Q, D = ck.ck_fp4_linear, ck.ck_fp4_expert_linear, ck.ck_quant_fp4, ck.ck_dequant_fp4

    def into(fn, shape, dt, *a, **kw):
        out = torch.full(shape, -3.0, dtype=dt, device="cuda")
        assert fn(*a, out=out, **kw) is out
        return out

    good = [
        lambda: Q(x, NV), lambda: Q(x, NV, tensor_scale=t), lambda: Q(x.float(), MX), lambda: Q(x[:0], NV),
        lambda: Q(x[:, :528], NV), lambda: Q(x[:1].half(), NV), lambda: Q(x[:, ::2], NV),
        lambda: D(codes, scales, NV), lambda: D(codes, scales, NV, tensor_scale=t, out_dtype=F32),
        lambda: D(codes[:1], scales, NV, out_dtype=F16), lambda: D(codes[:0], scales, NV),
        lambda: L(x, w, ws, NV), lambda: L(x[:1], w, ws, NV, bias), lambda: L(x[:0], w, ws, NV),
        lambda: L(x.float(), w, ws, NV, bias.bfloat16(), x_tensor_scale=t, w_tensor_scale=t),
        lambda: L(codes, w, ws, NV, x_scales=scales), lambda: L(codes, w, ws, NV, bias, x_scales=scales),
        lambda: L(codes[:1], w, ws, NV, x_scales=scales, out_dtype=F16), lambda: L(x, w[:1], ws, NV),
        lambda: L(x, w, ws, NV, workspace=work, dev_status=status), lambda: L(x, w, ws, NV, out_dtype=F32),
        lambda: into(L, (40, 200), F16, x, w, ws, NV), lambda: L(x.t().contiguous().t(), w, ws, NV),
        lambda: into(X, (40, 64), F32, x, off, w3, ws3, NV, bias3, w_tensor_scale=tw3),
        lambda: into(X, (40, 64), BF16, ecodes, off, w3, ws3, NV, x_scales=escales, x_tensor_scale=t),
    ]
    refused = [
        lambda: L(x, w[:, :16], ws, NV), lambda: L(x, w, ws[:-16], NV), lambda: L(x, w, ws, 9),
        lambda: L(x, w, ws, NV, bias[:-1]), lambda: L(x, w, ws, MX, x_tensor_scale=t),
        lambda: L(codes, w, ws, NV), lambda: L(x, w, ws, NV, out_dtype=torch.int32), lambda: L(x, w3, ws3, NV),
        lambda: L(x.cpu(), w, ws, NV), lambda: L(x, w, ws.cpu(), NV), lambda: L(x.int(), w, ws, NV),
        lambda: L(x, w, ws, NV, workspace=work[:-256]), lambda: L(x, w, ws, NV, out=bias),
        lambda: X(x, off.long(), w3, ws3, NV), lambda: X(x, off[:3], w3, ws3, NV), lambda: X(x, off, w, ws, NV),
        lambda: X(x, None, w3, ws3, NV), lambda: X(x, off, w3, ws3.flatten(), NV), lambda: Q(x[:, :40], NV),
        lambda: Q(x[0], NV), lambda: Q(x, NV, tensor_scale=t.double()), lambda: D(codes.char(), scales, NV),
        lambda: D(codes, scales[:-16], NV), lambda: D(codes, scales, NV, out_dtype=torch.int32),
    ]
    return good, refused


def test_native_and_python_host_sides_agree(monkeypatch):
    """The native host side takes every ordinary call, gives the bits that Python's way gives, and
    refuses what Python's way refuses, with its words."""
    assert ck._bind is not None, "_ck_bind is not built"
    good, refused = _forms()
    native = [f() for f in good]
    errors = []
    for f in refused:
        with pytest.raises(Exception) as e:
            f()
        errors.append(e)
    monkeypatch.setattr(ck, "_bind", None)
    for i, (f, n) in enumerate(zip(good, native)):
        p = f()
        for a, b in zip(n, p) if isinstance(p, tuple) else ((n, p),):
            assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(
                a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), f"form {i}"
    for i, (f, e) in enumerate(zip(refused, errors)):
        with pytest.raises(type(e.value)) as again:
            f()
        assert str(again.value) == str(e.value), f"refused form {i}"


def test_native_host_side_takes_ordinary_calls():
    x, w, ws = _case(NV, 20, 64, 128)
    codes, scales = ck._bind.quant(x, NV, None, None, None, None)
    assert isinstance(ck._bind.dequant(codes, scales, NV, None, None, BF16), torch.Tensor)
    out = ck._bind.product(x, None, w, ws, NV, None, None, None, None, None, None, None, None)
    assert torch.equal(out, ck.ck_fp4_linear(x, w, ws, NV))
    for bad in [(x.cpu(), NV), (x, 7), (x, None), (None, NV), (x.int(), NV), (x[:, :24], NV)]:
        assert ck._bind.quant(*bad, None, None, None, None) is None
    assert ck._bind.quant() is None and ck._bind.product(x) is None
