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


SHAPES = [(1, 1, 32), (1, 3840, 3840), (7, 200, 16384), (8, 96, 272), (9, 4000, 1040), (15, 333, 10240), (16, 129, 16400),
          (17, 130, 12320), (40, 200, 12304), (2, 40, 64), (5, 300, 96), (16, 130, 800), (31, 257, 1056),
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
