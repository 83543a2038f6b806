"""GPU tests of how the fp4 calls are made on the host: the first call of a host thread, several
threads at once, and after a call that failed."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess
import threading

import pytest
import torch

from rotated_w4a4_quantized_group_b200 import build as ck_build
from rotated_w4a4_quantized_group_b200 import ck
from rotated_w4a4_quantized_group_b200 import workloads as W
from test_fp4_gpu import BF16, FMT
from test_fp4_tiles_gpu import tile

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.lib()
    yield
    torch.cuda.synchronize()


def _linear(M, N, K, fmt, seed, codes=True):
    """A call of the C entry point on a stream handle, its output, and what it should be."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=g, dtype=BF16)
    w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
    want, out = ck.ck_fp4_linear(x, w, ws, fmt), torch.empty(M, N, dtype=BF16, device="cuda")
    work = torch.empty(max(ck.fp4_workspace_bytes(M, K, fmt), 1), dtype=torch.uint8, device="cuda")
    dt, sm, xs = ck.CK_BF16, K, None
    if codes:
        x, xs = ck.ck_quant_fp4(x, fmt)
        dt, sm = ck.CK_FP4, x.stride(0)
    fn = ck.lib().ck_fp4_linear

    def call(stream, keep=(x, xs, w, ws, work)):
        return fn(x.data_ptr(), dt, M, K, sm, 1, fmt, None if xs is None else xs.data_ptr(), None, w.data_ptr(), N,
                  w.stride(0), ws.data_ptr(), None, None, 0, out.data_ptr(), ck.CK_BF16, N, work.data_ptr(),
                  work.numel(), None, stream)

    return call, out, want


def _in_a_new_thread(f):
    got = []

    def go():
        try:
            got.append(f())
        except Exception as e:
            got.append(e)

    t = threading.Thread(target=go)
    t.start()
    t.join()
    return got[0]


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b)) if isinstance(a, tuple) else torch.equal(a, b)


@FMT
@pytest.mark.parametrize("M", [4, 40, 400, 3000])
def test_the_first_call_of_a_host_thread(fmt, M):
    """A thread that has made no CUDA call: its allocations are served from memory that is there, so that the
    library's call is its first."""
    N, K = 1600, 512
    g = torch.Generator(device="cuda").manual_seed(160)
    x = torch.randn(M, K, device="cuda", generator=g, dtype=BF16)
    w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
    codes, scales = ck.ck_quant_fp4(x, fmt)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    calls = [lambda: ck.ck_fp4_linear(x, w, ws, fmt), lambda: ck.ck_fp4_linear(codes, w, ws, fmt, x_scales=scales),
             lambda: ck.ck_quant_fp4(x, fmt), lambda: ck.ck_dequant_fp4(codes, scales, fmt),
             lambda: ck.ck_fp4_expert_linear(codes, off, w[None], ws[None], fmt,
                                             x_scales=ck.ck_quant_fp4(x, fmt, offsets=off)[1])]
    for i, f in enumerate(calls):
        want = f()
        del want                      # the allocator keeps its memory
        want = f()
        torch.cuda.synchronize()
        got = _in_a_new_thread(f)
        assert not isinstance(got, Exception), f"call {i}: {got}"
        assert _same(got, want), f"call {i}"
    call, out, want = _linear(M, N, K, fmt, 161)
    torch.cuda.synchronize()
    handle = torch.cuda.current_stream().cuda_stream
    assert _in_a_new_thread(lambda: call(handle)) == ck.CK_OK
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("M", [40, 300])
def test_the_first_int4_call_of_a_host_thread(M):
    case = W.LINEAR_CASES[W.HEADLINE].replace(M=M, N=320, K=448)
    inp = {k: v.cuda() if torch.is_tensor(v) else v for k, v in W.make_linear_inputs(case).items()}

    def f():
        return ck.ck_w4a4_linear(inp["x"], inp["R"], case.g, inp["w_packed"], inp["w_scale"], inp["bias"])

    want = f()
    del want
    want = f()
    torch.cuda.synchronize()
    got = _in_a_new_thread(f)
    assert not isinstance(got, Exception), got
    assert torch.equal(got, want)


HAMMER = r"""
#include <thread>
#include "ck.h"
// One thread per call: the call again and again, on a stream of its own; returns how many did not return CK_OK.
struct Call {
    const void* x; long long M, K, sm; int fmt; const unsigned char* xs; const unsigned char* w; long long N, w_ld;
    const unsigned char* ws; void* out; cudaStream_t stream; int bad;
};
extern "C" void hammer(decltype(&ck_fp4_linear) fn, Call* c, int n, int times) {
    std::thread t[8];
    for (int i = 0; i < n; ++i)
        t[i] = std::thread([=] {
            for (int k = 0; k < times; ++k)
                c[i].bad += fn(c[i].x, CK_FP4, c[i].M, c[i].K, c[i].sm, 1, (ck_fp4_format)c[i].fmt, c[i].xs, nullptr,
                               c[i].w, c[i].N, c[i].w_ld, c[i].ws, nullptr, nullptr, CK_F32, c[i].out, CK_BF16, c[i].N,
                               nullptr, 0, nullptr, c[i].stream) != CK_OK;
        });
    for (int i = 0; i < n; ++i) t[i].join();
}
"""


class _Call(ctypes.Structure):
    _fields_ = [(n, t) for n, t in zip(
        ("x", "M", "K", "sm", "fmt", "xs", "w", "N", "w_ld", "ws", "out", "stream", "bad"),
        (ctypes.c_void_p, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p,
         ctypes.c_void_p, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
         ctypes.c_int))]


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    d = tmp_path_factory.mktemp("hammer")
    (d / "hammer.cpp").write_text(HAMMER)
    cuda = os.path.join(os.path.dirname(os.path.dirname(ck_build.nvcc())), "include")
    subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-pthread", "-I" + cuda,
                    "-I" + ck_build.INCLUDE, str(d / "hammer.cpp"), "-o", str(d / "hammer.so")], check=True)
    return ctypes.CDLL(str(d / "hammer.so")).hammer


@FMT
@pytest.mark.parametrize("tiles,shapes", [(((0, 64), (0, 64)), ((33, 128, 2048), (33, 128, 12288))),
                                          (((1, 64), (1, 128)), ((400, 1600, 1024), (900, 2100, 768)))],
                         ids=["few tiles", "one CTA a tile"])
def test_host_threads_with_different_sizes(hammer, fmt, tiles, shapes):
    """Two threads launch one kernel with different amounts of shared memory: neither takes the other's
    allowance away between its being set and the launch."""
    for t, s in zip(tiles, shapes):
        ctas, rows = tile(*s, fmt)
        assert ctas == t[0] and (ctas == 0 or rows == t[1])
    calls, keep = (_Call * 2)(), []
    for i, (M, N, K) in enumerate(shapes):
        g = torch.Generator(device="cuda").manual_seed(140 + i)
        x, xs = ck.ck_quant_fp4(torch.randn(M, K, device="cuda", generator=g), fmt)
        w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
        out, stream = torch.empty(M, N, dtype=BF16, device="cuda"), torch.cuda.Stream()
        keep.append((x, xs, w, ws, out, stream, ck.ck_fp4_linear(x, w, ws, fmt, x_scales=xs, out_dtype=BF16)))
        calls[i] = _Call(x.data_ptr(), M, K, x.stride(0), fmt, xs.data_ptr(), w.data_ptr(), N, w.stride(0),
                         ws.data_ptr(), out.data_ptr(), stream.cuda_stream, 0)
    torch.cuda.synchronize()
    hammer(ctypes.cast(ck.lib().ck_fp4_linear, ctypes.c_void_p), calls, 2, 50000)
    torch.cuda.synchronize()
    assert [c.bad for c in calls] == [0, 0]
    for *_, out, _, want in keep:
        assert torch.equal(out, want)


@FMT
@pytest.mark.parametrize("M", [4, 40, 100, 3000])
def test_a_failed_call_is_not_the_next_ones_fault(fmt, M):
    """A launch into a capture that something else has ended fails on the host; the next call, elsewhere, is
    right and says so."""
    call, out, want = _linear(M, 907, 4096, fmt, 150, M > 16)
    x = torch.randn(64, 128, device="cuda", dtype=BF16)
    cudart = ctypes.CDLL("libcudart.so.12")
    stream = torch.cuda.Stream()
    handle = ctypes.c_void_p(stream.cuda_stream)
    for after in (lambda: call(torch.cuda.current_stream().cuda_stream), lambda: ck.ck_quant_fp4(x, fmt) and ck.CK_OK):
        torch.cuda.synchronize()
        assert cudart.cudaStreamBeginCapture(handle, 2) == 0             # relaxed
        assert cudart.cudaStreamSynchronize(handle) != 0                 # not allowed there: the capture is void
        failed = call(stream.cuda_stream)
        graph = ctypes.c_void_p()
        assert cudart.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
        cudart.cudaGetLastError()
        assert failed == ck.CK_ERR_CUDA
        assert after() == ck.CK_OK
    assert call(torch.cuda.current_stream().cuda_stream) == ck.CK_OK
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_negated_views_are_refused_on_both_host_sides(monkeypatch):
    M, N, K = 20, 64, 128
    g = torch.Generator(device="cuda").manual_seed(170)
    z = torch.randn(M, K, 2, device="cuda", generator=g)
    plain, neg = torch.view_as_complex(z).imag, torch.view_as_complex(z).conj().imag
    w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g), ck.CK_NVFP4)
    t = torch.view_as_complex(torch.ones(1, 2, device="cuda")).conj().imag
    calls = [lambda v: ck.ck_quant_fp4(v, ck.CK_NVFP4)[0], lambda v: ck.ck_fp4_linear(v, w, ws, ck.CK_NVFP4)]
    for bind in (ck._bind, None):
        monkeypatch.setattr(ck, "_bind", bind)
        for f in calls:
            with pytest.raises(ValueError, match="negated view"):
                f(neg)
            assert torch.equal(f(neg.resolve_neg()), f(-plain)) and torch.equal(f(plain), f(plain.contiguous()))
        with pytest.raises(ValueError, match="negated view"):
            ck.ck_quant_fp4(plain, ck.CK_NVFP4, tensor_scale=t)
