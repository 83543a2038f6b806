"""GPU tests of how the fp4 calls are made on the host: the first call of a host thread, several
threads at once, and after a call that failed."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

from rotated_w4a4_quantized_group_b200 import ck
from rotated_w4a4_quantized_group_b200 import workloads as W
from test_fp4_gpu import BF16, FMT

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
