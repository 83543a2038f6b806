"""The host side of the fp4 calls where no GPU is needed: what ck.py hands to the library, and what it
refuses.  Its launch is replaced by a record of the arguments, its device check by one that takes host
tensors; nothing is launched."""
from __future__ import annotations

import subprocess
import warnings

import pytest
import torch

from rotated_w4a4_quantized_group_b200 import build as ck_build
from rotated_w4a4_quantized_group_b200 import ck

MX, NV = ck.CK_MXFP4, ck.CK_NVFP4
BOTH = pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])


@pytest.fixture
def launched(monkeypatch):
    """The (entry point, arguments) that reach the library."""
    ck_build.build()
    ck.lib()
    calls = []
    monkeypatch.setattr(ck, "_bind", None)
    monkeypatch.setattr(ck, "_on_device", lambda x, *ts: 0)
    monkeypatch.setattr(ck, "_launch", lambda name, dev, args: calls.append((name, args)))
    return calls


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


# ------------------------------------------------------------------- rows that overlap

def _overlapping(fmt):
    """Calls with a tensor whose rows lie on top of one another: walked at a pitch of whole rows, it would
    lead past its memory."""
    M, N, K = 8, 24, 128
    x, codes, w = torch.zeros(M, K), _u8(M, K // 2), _u8(N, K // 2)
    sx, sw = _u8(ck.fp4_scales_bytes(M, K, fmt)), _u8(ck.fp4_scales_bytes(N, K, fmt))
    off = torch.tensor([0, 3, M], dtype=torch.int32)
    sx2 = _u8(ck.fp4_scales_bytes(M, K, fmt, 2))
    for row in (lambda r, c, dt=torch.uint8: torch.zeros(1, c, dtype=dt).expand(r, c),
                lambda r, c, dt=torch.uint8: torch.zeros(r * c, dtype=dt).as_strided((r, c), (c - 1, 1))):
        out = row(M, N, torch.float32)
        yield "codes", lambda: ck.ck_quant_fp4(x, fmt, codes=row(M, K // 2))
        yield "codes", lambda: ck.ck_dequant_fp4(row(M, K // 2), sx, fmt)
        yield "out", lambda: ck.ck_dequant_fp4(codes, sx, fmt, out=row(M, K, torch.float32))
        yield "x", lambda: ck.ck_fp4_linear(row(M, K // 2), w, sw, fmt, x_scales=sx)
        yield "w_codes", lambda: ck.ck_fp4_linear(x, row(N, K // 2), sw, fmt)
        yield "out", lambda: ck.ck_fp4_linear(x, w, sw, fmt, out=out)
        yield "x", lambda: ck.ck_fp4_expert_linear(row(M, K // 2), off, _u8(2, N, K // 2), torch.stack([sw, sw]), fmt,
                                                   x_scales=sx2)
        yield "w_codes", lambda: ck.ck_fp4_expert_linear(x, off, torch.stack([w, w])[:, :1].expand(2, N, K // 2),
                                                         torch.stack([sw, sw]), fmt)
        yield "out", lambda: ck.ck_fp4_expert_linear(x, off, torch.stack([w, w]), torch.stack([sw, sw]), fmt, out=out)


@BOTH
def test_overlapping_rows_are_refused(launched, fmt):
    for what, call in _overlapping(fmt):
        with pytest.raises(ValueError, match=f"{what}'s rows must not overlap"):
            call()
    assert not launched


@BOTH
def test_a_single_rows_pitch_is_not_used(launched, fmt):
    K, N = 128, 24
    w, sw, sx = _u8(N, K // 2), _u8(ck.fp4_scales_bytes(N, K, fmt)), _u8(ck.fp4_scales_bytes(1, K, fmt))
    codes, out = _u8(K // 2).expand(1, K // 2), torch.zeros(N).expand(1, N)
    ck.ck_quant_fp4(torch.zeros(1, K), fmt, codes=codes)
    ck.ck_dequant_fp4(codes, sx, fmt, out=torch.zeros(K).expand(1, K))
    ck.ck_fp4_linear(codes, w, sw, fmt, x_scales=sx, out=out)
    ck.ck_fp4_linear(torch.zeros(1, K), w[:1], sw, fmt)
    names = [name for name, _ in launched]
    assert names == ["ck_quant_fp4", "ck_dequant_fp4", "ck_fp4_linear", "ck_fp4_linear"]
    for ldq in (launched[0][1][11], launched[1][1][1], launched[2][1][4], launched[3][1][11]):
        assert ldq == K // 2


# ------------------------------------------------------------------- values that are not in memory

def test_negated_views_are_refused(launched):
    """The imaginary part of a conjugate is a view whose memory holds the negatives of its values."""
    def neg(*shape):
        t = torch.view_as_complex(torch.ones(*shape, 2)).conj().imag
        assert t.is_neg() and t.dtype == torch.float32
        return t

    M, N, K = 4, 24, 128
    x, w, sw = torch.zeros(M, K), _u8(N, K // 2), _u8(ck.fp4_scales_bytes(N, K, NV))
    codes, sx, t = _u8(M, K // 2), _u8(ck.fp4_scales_bytes(M, K, NV)), torch.ones(1)
    for what, call in [
            ("x", lambda: ck.ck_quant_fp4(neg(M, K), NV)),
            ("tensor_scale", lambda: ck.ck_quant_fp4(x, NV, tensor_scale=neg(1))),
            ("tensor_scale", lambda: ck.ck_dequant_fp4(codes, sx, NV, tensor_scale=neg(1))),
            ("x", lambda: ck.ck_fp4_linear(neg(M, K), w, sw, NV)),
            ("bias", lambda: ck.ck_fp4_linear(x, w, sw, NV, neg(N))),
            ("x_tensor_scale", lambda: ck.ck_fp4_linear(x, w, sw, NV, x_tensor_scale=neg(1))),
            ("w_tensor_scale", lambda: ck.ck_fp4_linear(x, w, sw, NV, x_tensor_scale=t, w_tensor_scale=neg(1))),
            ("x", lambda: ck.ck_fp4_expert_linear(neg(M, K), torch.zeros(2, dtype=torch.int32), w[None], sw[None], NV))]:
        with pytest.raises(ValueError, match=f"{what} is a negated view"):
            call()
    assert not launched


# ------------------------------------------------------------------- limits

@BOTH
@pytest.mark.parametrize("M,K,E", [(2 ** 31 - 1, 128 * 130, 0), (2 ** 24 * 128 - 1, 128 * 128, 0),
                                   (2 ** 24 * 128 - 128 * 1000, 128 * 128, 1000), (2 ** 30, 2 ** 15, 0)])
def test_more_tiles_than_a_grid_are_refused(fmt, M, K, E):
    """2^31 tiles of 128 x 128 and a few more, which are about half as many of 128 x 256."""
    ck_build.build()
    L, P = ck.lib(), 1 << 20
    rows = M // 128 + E if E else -(-M // 128)
    assert 2 ** 31 <= rows * (K // 128) < 1.02 * 2 ** 31
    off = P if E else None
    assert L.ck_quant_fp4(P, ck.CK_BF16, M, K, K, 1, fmt, None, off, E, P, K // 2, P, None) == ck.CK_ERR_UNSUPPORTED
    assert L.ck_dequant_fp4(P, K // 2, P, M, K, fmt, None, off, E, P, ck.CK_BF16, K, None) == ck.CK_ERR_UNSUPPORTED


@BOTH
def test_more_channels_than_few_rows_take_are_refused(fmt):
    """Rows quantized inside: 65535 tiles of 128 channels."""
    ck_build.build()
    L, P = ck.lib(), 1 << 20
    N = 65535 * 128 + 1
    for M, K in ((1, 64), (16, 2048)):
        assert L.ck_fp4_linear(P, ck.CK_BF16, M, K, K, 1, fmt, None, None, P, N, K // 2, P, None, None, 0, P, ck.CK_BF16, N,
                               None, 0, None, None) == ck.CK_ERR_UNSUPPORTED


# ------------------------------------------------------------------- addresses

ODD = [("quant", dict(x=1)), ("quant", dict(dt=ck.CK_F32, x=2)), ("quant", dict(ts=2)), ("quant", dict(off=2, E=2)),
       ("dequant", dict(out=1)), ("dequant", dict(odt=ck.CK_F32, out=2)), ("dequant", dict(ts=1)),
       ("dequant", dict(off=2, E=2)), ("linear", dict(x=1)), ("linear", dict(dt=ck.CK_F32, x=2)), ("linear", dict(out=1)),
       ("linear", dict(odt=ck.CK_F32, out=2)), ("linear", dict(bias=2)), ("linear", dict(bdt=ck.CK_F16, bias=1)),
       ("linear", dict(xts=2)), ("linear", dict(wts=2)), ("linear", dict(status=2)), ("linear", dict(M=4, x=1)),
       ("experts", dict(off=2)), ("experts", dict(wts=1)), ("experts", dict(out=1)), ("experts", dict(status=1))]


@pytest.mark.parametrize("fn,odd", ODD)
def test_addresses_that_no_element_has_are_refused(fn, odd):
    """A pointer that is not a multiple of its type's size would be a misaligned access on the device."""
    ck_build.build()
    L, P = ck.lib(), 1 << 20
    a = dict(x=0, dt=ck.CK_BF16, M=40, E=3, off=None, ts=None, out=0, odt=ck.CK_BF16, xts=None, wts=None, bias=None,
             bdt=ck.CK_F32, status=None)
    a.update(odd)
    at = {k: None if a[k] is None else P + a[k] for k in ("x", "off", "ts", "out", "xts", "wts", "bias", "status")}
    if fn == "quant":
        st = L.ck_quant_fp4(at["x"], a["dt"], a["M"], 64, 64, 1, NV, at["ts"], at["off"], a["E"], P, 32, P, None)
    elif fn == "dequant":
        st = L.ck_dequant_fp4(P, 32, P, a["M"], 64, NV, at["ts"], at["off"], a["E"], at["out"], a["odt"], 64, None)
    else:
        head = (at["x"], a["dt"], a["M"], 64, 64, 1, NV, None, at["xts"])
        tail = (P, at["wts"], at["bias"], a["bdt"], at["out"], a["odt"], 8, P, 1 << 20, at["status"], None)
        if fn == "linear":
            st = L.ck_fp4_linear(*head, P, 8, 32, *tail)
        else:
            st = L.ck_fp4_expert_linear(*head, P if at["off"] is None else at["off"], 3, P, 8, 32, 256, *tail)
    assert st == ck.CK_ERR_INVALID_ARG


# ------------------------------------------------------------------- the native host side's torch

@pytest.fixture
def bind(monkeypatch):
    ck_build.build_all()
    monkeypatch.setattr(ck, "_lib", None)
    monkeypatch.setattr(ck, "_bind", None)
    from rotated_w4a4_quantized_group_b200 import _ck_bind
    return _ck_bind


def test_the_native_host_side_serves_the_torch_it_was_built_for(bind):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        ck.lib()
    assert bind.torch_version == torch.__version__ and ck._bind is bind


def test_the_native_host_side_is_left_out_with_another_torch(bind, monkeypatch):
    monkeypatch.setattr(bind, "torch_version", "0.1")
    with pytest.warns(UserWarning, match="built against torch 0.1"):
        ck.lib()
    assert ck._bind is None


def test_the_native_host_side_is_built_again_for_another_torch(bind, monkeypatch, tmp_path):
    """With a file for the extension that is newer than its sources."""
    so, runs = tmp_path / "_ck_bind.so", []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(ck_build, "BIND", str(so))
    monkeypatch.setattr(ck_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(ck_build.subprocess, "run", run)
    for version, builds in ((torch.__version__, 1), (torch.__version__, 1), ("9.9", 2), ("9.9", 2), ("9.8", 3)):
        monkeypatch.setattr(torch, "__version__", version)
        ck_build.build_bind()
        assert len(runs) == builds and so.exists()
        assert f'-DCK_TORCH_VERSION="{version}"' in runs[-1]


# ------------------------------------------------------------------- counts of tiles

COUNTS = r"""
#include <cstdio>
#include <vector>
#include "ck_fp4.cuh"
// experts' counts, lines of "n c0 c1 ...", added up in order and as a tree; then what the units take of them
int main() {
    int n;
    while (std::scanf("%d", &n) == 1) {
        std::vector<int> c(n);
        for (int& v : c) std::scanf("%d", &v);
        int sum = 0;
        for (int v : c) sum = ck::tiles_add(sum, v);
        std::vector<int> t = c;
        for (size_t d = 1; d < t.size(); d *= 2)
            for (size_t i = 0; i + d < t.size(); i += 2 * d) t[i] = ck::tiles_add(t[i], t[i + d]);
        unsigned long long taken = 0;
        unsigned last = 0;
        for (int u = 0; u < 148; ++u) {
            const unsigned k = ck::tiles_of_unit(sum, u, 148);
            taken += k;
            if (k && u + (k - 1) * 148ull > last) last = u + (k - 1) * 148ull;
        }
        std::printf("%d %d %llu %u\n", sum, t[0], taken, last);
    }
}
"""


def test_counts_of_tiles_never_wrap(tmp_path):
    """Offsets that decrease can give half of the experts all the rows: the sum stays an int, and the units
    take each tile once, none behind the last."""
    src, exe = tmp_path / "counts.cu", tmp_path / "counts"
    src.write_text(COUNTS)
    subprocess.run([ck_build.nvcc(), "-std=c++17", "-I" + ck_build.INCLUDE, "-I" + ck_build.CSRC, *ck_build.ARCH,
                    "-o", str(exe), str(src)], check=True)
    top = 2 ** 31 - 1
    cases = [[5, 0, 7], [0], [1] * 300, [1024 * 4096, 0] * 512, [top], [top, 1], [1, top, top], [top - 1, 1, 0],
             [2 ** 30, 2 ** 30], [2 ** 30, 2 ** 30 - 1, 0, 3]]
    text = "".join(f"{len(c)} {' '.join(map(str, c))}\n" for c in cases)
    got = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for c, line in zip(cases, got):
        want = min(sum(c), top)
        assert [int(v) for v in line.split()] == [want, want, want, max(want - 1, 0)], c


# ------------------------------------------------------------------- the tests' own reach

@BOTH
def test_shapes_of_the_tile_tests_get_their_tiles(fmt):
    """The GPU tests of one tile shape reach it by the library's rule, here too, where a change of the rule
    shows at once."""
    import test_fp4_tiles_gpu as t

    ck_build.build()
    for want, M, N, K in t.LINEARS:
        for ragged in (False, True):
            assert t.tile(M, N, t.width(K, fmt), fmt, ragged=ragged) == want, (M, N, K)
    for want, off, N, K in t.EXPERTS:
        assert t.tile(off[-1] + 9, N, t.width(K, fmt), fmt, len(off) - 1) == want, (off, N, K)
