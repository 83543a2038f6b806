"""The fp4 entry points reject invalid calls on the host, before any CUDA work (no device needed),
and so does their binding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp4_ref as ref
from rotated_w4a4_quantized_group_b200 import build as ck_build
from rotated_w4a4_quantized_group_b200 import ck

MX, NV = ck.CK_MXFP4, ck.CK_NVFP4
P, NULL = 1 << 20, None
BOTH = pytest.mark.parametrize("fmt", [MX, NV])


@pytest.fixture(scope="module")
def L():
    ck_build.build()
    return ck.lib()


def quant(L, **kw):
    a = dict(x=P, dt=ck.CK_BF16, M=4, K=64, sm=64, sk=1, fmt=NV, ts=NULL, off=NULL, E=0, codes=P, ldq=32,
             scales=P)
    a.update(kw)
    return L.ck_quant_fp4(a["x"], a["dt"], a["M"], a["K"], a["sm"], a["sk"], a["fmt"], a["ts"], a["off"],
                          a["E"], a["codes"], a["ldq"], a["scales"], None)


BAD_QUANT = [dict(dt=ck.CK_I8), dict(dt=ck.CK_FP4), dict(dt=9), dict(M=-1), dict(K=0), dict(K=-32),
             dict(K=40), dict(fmt=MX, K=48), dict(fmt=2), dict(fmt=-1), dict(ldq=31), dict(fmt=MX, ts=P),
             dict(off=P, E=0), dict(off=P, E=1025), dict(off=P, E=-1), dict(x=NULL), dict(codes=NULL),
             dict(scales=NULL), dict(scales=P + 8)]


@pytest.mark.parametrize("bad", BAD_QUANT)
def test_quant_rejects_on_host(L, bad):
    assert quant(L, **bad) == ck.CK_ERR_INVALID_ARG


def test_quant_sizes_it_does_not_take(L):
    assert quant(L, M=1 << 31) == ck.CK_ERR_UNSUPPORTED
    assert quant(L, K=1 << 31, ldq=1 << 30) == ck.CK_ERR_UNSUPPORTED
    assert quant(L, M=(1 << 31) - 1, K=(1 << 31) - 32, ldq=1 << 30) == ck.CK_ERR_UNSUPPORTED


def test_empty_calls_are_no_ops(L):
    assert quant(L, M=0, x=NULL, codes=NULL, scales=NULL) == ck.CK_OK
    assert dequant(L, M=0, codes=NULL, scales=NULL, out=NULL) == ck.CK_OK
    assert linear(L, M=0, x=NULL, out=NULL, ws=NULL, wsb=0) == ck.CK_OK
    assert linear(L, N=0, ldo=0, w=NULL, wsc=NULL, out=NULL, ws=NULL, wsb=0) == ck.CK_OK
    assert experts(L, M=0, x=NULL, off=NULL, out=NULL, ws=NULL, wsb=0) == ck.CK_OK


def dequant(L, **kw):
    a = dict(codes=P, ldq=32, scales=P, M=4, K=64, fmt=NV, ts=NULL, off=NULL, E=0, out=P, odt=ck.CK_BF16,
             ldo=64)
    a.update(kw)
    return L.ck_dequant_fp4(a["codes"], a["ldq"], a["scales"], a["M"], a["K"], a["fmt"], a["ts"], a["off"],
                            a["E"], a["out"], a["odt"], a["ldo"], None)


@pytest.mark.parametrize("bad", [dict(odt=ck.CK_I8), dict(odt=ck.CK_FP4), dict(M=-1), dict(K=0), dict(K=40),
                                 dict(fmt=MX, K=48), dict(fmt=7), dict(ldq=31), dict(ldo=63),
                                 dict(fmt=MX, ts=P), dict(off=P, E=0), dict(codes=NULL), dict(scales=NULL),
                                 dict(out=NULL), dict(scales=P + 4)])
def test_dequant_rejects_on_host(L, bad):
    assert dequant(L, **bad) == ck.CK_ERR_INVALID_ARG


def linear(L, **kw):
    a = dict(x=P, dt=ck.CK_BF16, M=40, K=64, sm=64, sk=1, fmt=NV, xs=NULL, xts=NULL, w=P, N=8, w_ld=32, wsc=P,
             wts=NULL, bias=NULL, bdt=ck.CK_F32, out=P, odt=ck.CK_BF16, ldo=8, ws=P, wsb=1 << 20)
    a.update(kw)
    return L.ck_fp4_linear(a["x"], a["dt"], a["M"], a["K"], a["sm"], a["sk"], a["fmt"], a["xs"], a["xts"],
                           a["w"], a["N"], a["w_ld"], a["wsc"], a["wts"], a["bias"], a["bdt"], a["out"],
                           a["odt"], a["ldo"], a["ws"], a["wsb"], None, None)


CODES = dict(dt=ck.CK_FP4, sm=32, xs=P)
BAD_LINEAR = [dict(dt=ck.CK_I8), dict(dt=7), dict(odt=ck.CK_FP4), dict(odt=ck.CK_I8), dict(M=-1), dict(N=-1),
              dict(K=0), dict(K=40), dict(fmt=MX, K=48), dict(fmt=3), dict(w_ld=31), dict(w_ld=40),
              dict(ldo=7), dict(x=NULL), dict(w=NULL), dict(wsc=NULL), dict(out=NULL), dict(w=P + 8),
              dict(wsc=P + 8), dict(fmt=MX, xts=P), dict(fmt=MX, wts=P), dict(bias=P, bdt=ck.CK_I8),
              dict(CODES, xs=NULL), dict(CODES, sk=2), dict(CODES, sm=31), dict(CODES, sm=40),
              dict(CODES, x=P + 8), dict(CODES, xs=P + 8)]


@pytest.mark.parametrize("bad", BAD_LINEAR)
def test_linear_rejects_on_host(L, bad):
    assert linear(L, **bad) == ck.CK_ERR_INVALID_ARG


def test_linear_workspace(L):
    assert linear(L, ws=NULL, wsb=0) == ck.CK_ERR_WORKSPACE
    assert linear(L, wsb=100) == ck.CK_ERR_WORKSPACE
    assert linear(L, ws=P + 16) == ck.CK_ERR_WORKSPACE
    assert linear(L, M=1 << 31) == ck.CK_ERR_UNSUPPORTED
    assert linear(L, N=1 << 31, ldo=1 << 31) == ck.CK_ERR_UNSUPPORTED


def experts(L, **kw):
    a = dict(x=P, dt=ck.CK_BF16, M=40, K=64, sm=64, sk=1, fmt=NV, xs=NULL, xts=NULL, off=P, E=3, w=P, N=8,
             w_ld=32, w_stride=256, wsc=P, wts=NULL, bias=NULL, bdt=ck.CK_F32, out=P, odt=ck.CK_BF16, ldo=8,
             ws=P, wsb=1 << 20)
    a.update(kw)
    return L.ck_fp4_expert_linear(a["x"], a["dt"], a["M"], a["K"], a["sm"], a["sk"], a["fmt"], a["xs"],
                                  a["xts"], a["off"], a["E"], a["w"], a["N"], a["w_ld"], a["w_stride"],
                                  a["wsc"], a["wts"], a["bias"], a["bdt"], a["out"], a["odt"], a["ldo"],
                                  a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("bad", BAD_LINEAR + [dict(off=NULL), dict(E=0), dict(E=-1), dict(E=1025),
                                              dict(w_stride=255), dict(w_stride=240), dict(w_stride=-256)])
def test_expert_linear_rejects_on_host(L, bad):
    assert experts(L, **bad) == ck.CK_ERR_INVALID_ARG


def test_expert_linear_workspace(L):
    assert experts(L, ws=NULL, wsb=0) == ck.CK_ERR_WORKSPACE
    assert experts(L, wsb=ck.fp4_workspace_bytes(40, 64, NV, 3) - 1) == ck.CK_ERR_WORKSPACE


@BOTH
@pytest.mark.parametrize("M,K", [(1, 32), (128, 64), (129, 96), (300, 4128)])
def test_scale_and_workspace_sizes(L, fmt, M, K):
    b = ref.BLOCK[fmt]
    tiles = -(-(K // b) // 4)
    assert ck.fp4_scales_bytes(M, K, fmt) == -(-M // 128) * tiles * 512
    assert ck.fp4_scales_bytes(M, K, fmt, 7) == (M // 128 + 7) * tiles * 512
    assert ck.fp4_workspace_bytes(M, K, fmt, 7) >= M * (K // 2) + ck.fp4_scales_bytes(M, K, fmt, 7)
    if M > 16:
        assert ck.fp4_workspace_bytes(M, K, fmt) >= M * (K // 2) + ck.fp4_scales_bytes(M, K, fmt)


def test_sizes_of_invalid_arguments_are_zero(L):
    for a in [(-1, 64, NV, 0), (4, 40, NV, 0), (4, 48, MX, 0), (4, 64, 2, 0), (4, 64, NV, -1),
              (4, 64, NV, 1025), (1 << 31, 64, NV, 0), (4, 1 << 31, NV, 0)]:
        assert L.ck_fp4_scales_bytes(*a) == 0 and L.ck_fp4_linear_workspace_bytes(*a) == 0


def test_experts_scale_blocks_never_overlap():
    """Expert e's scales start at tile row offsets[e] / 128 + e: disjoint, and within the size given."""
    g = np.random.default_rng(0)
    for _ in range(200):
        E = int(g.integers(1, 12))
        off = np.sort(g.integers(0, 700, E + 1))
        used = set()
        for e in range(E):
            n = off[e + 1] - off[e]
            mine = set(range(off[e] // 128 + e, off[e] // 128 + e + -(-n // 128)))
            assert not used & mine
            used |= mine
        assert not used or max(used) < off[-1] // 128 + E


def test_binding_refuses_bad_tensors(L):
    """Shapes, types and host tensors are refused before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, ws = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        ck.ck_quant_fp4(x, NV)
    with pytest.raises(ValueError, match="CUDA device"):
        ck.ck_dequant_fp4(w, ws, NV)
    with pytest.raises(ValueError, match="CUDA device"):
        ck.ck_fp4_linear(x, w, ws, NV)
    with pytest.raises(ValueError, match="multiple of the block"):
        ck.ck_quant_fp4(x[:, :40], NV)
    with pytest.raises(ValueError, match="fmt"):
        ck.ck_quant_fp4(x, 5)
    with pytest.raises(ValueError, match="fp32, fp16 or bf16"):
        ck.ck_quant_fp4(x.to(torch.int8), NV)
    with pytest.raises(ValueError, match=r"\(N, K/2\)"):
        ck.ck_fp4_linear(x, w[None], ws, NV)
    with pytest.raises(ValueError, match="offsets"):
        ck.ck_fp4_expert_linear(x, None, w[None], ws[None], NV)


def test_reference_rounds_to_the_nearest():
    """The float64 reference itself: every code of E2M1 and E4M3 is a fixed point, borders go to the even
    code, and the nearest entry is within half a step."""
    for table in (ref.GRID, ref.E4M3):
        assert (ref.nearest(table, table) == np.arange(len(table))).all()
        mid = (table[1:] + table[:-1]) / 2
        n = ref.nearest(mid, table)
        assert (n % 2 == 0).all() and (np.abs(table[n] - mid) == (table[1:] - table[:-1]) / 2).all()
        q = np.random.default_rng(1).uniform(0, table[-1], 2000)
        assert (np.abs(table[ref.nearest(q, table)] - q) <= np.abs(table[None, :] - q[:, None]).min(1)).all()
