"""The native binding's checks that need no GPU: tensors that claim to lie on
one (PyTorch's fake tensors) are refused before their memory is asked for. And
what of det_gemm's binding does not depend on it."""
import os
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def dg():
    from invariant_deterministic_gemm_gb300 import _build
    _build.build()
    import invariant_deterministic_gemm_gb300 as m
    m.lib()
    return m


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="a fake tensor of cuda:1 needs none or two GPUs")
def test_tensors_of_different_devices_are_refused(dg):
    with FakeTensorMode():
        def t(dtype, *shape, device="cuda:0"):
            return torch.empty(shape, dtype=dtype, device=device)
        f32, i32, bf16, e4m3, far = torch.float32, torch.int32, torch.bfloat16, torch.float8_e4m3fn, dict(device="cuda:1")
        calls = [
            lambda: dg.det_moe_route(t(f32, 4, 8), 2, bias=t(f32, 8, **far)),
            lambda: dg.det_moe_route_bwd(t(f32, 4, 2, **far), t(f32, 4, 8), t(i32, 4, 2)),
            lambda: dg.det_moe_gather(t(bf16, 4, 64), t(i32, 8, **far), 2),
            lambda: dg.det_moe_gather(t(bf16, 4, 64), t(i32, 8), 2, out=t(bf16, 8, 64, **far)),
            lambda: dg.det_moe_combine(t(bf16, 8, 64), t(i32, 4, 2), t(f32, 4, 2, **far)),
            lambda: dg.det_moe_combine_bwd(t(bf16, 4, 64), t(bf16, 8, 64), t(i32, 8), t(i32, 4, 2, **far), t(f32, 4, 2)),
            lambda: dg.det_fp8_quantize_rows(t(bf16, 4, 64), t(i32, 8, **far), 2),
            lambda: dg.det_fp8_quantize_cols(t(bf16, 4, 64), t(i32, 3, **far)),
            lambda: dg.det_fp8_gemm(t(e4m3, 4, 128), t(f32, 4, 1), t(e4m3, 32, 128, **far), t(f32, 1, 1)),
            lambda: dg.det_fp8_gemm(t(e4m3, 4, 128), t(f32, 4, 1, **far), t(e4m3, 32, 128), t(f32, 1, 1)),
            lambda: dg.det_fp8_gemm_grouped(t(e4m3, 4, 128), t(f32, 4, 1), t(e4m3, 2, 32, 128), t(f32, 2, 1, 1), t(i32, 3, **far)),
            lambda: dg.det_fp8_gemm_wgrad(t(e4m3, 32, 128), t(f32, 1, 32), t(e4m3, 64, 128, **far), t(f32, 1, 64)),
            lambda: dg.det_embedding(t(i32, 4), t(bf16, 10, 64, **far)),
            lambda: dg.det_embedding_grad(t(bf16, 4, 64), t(i32, 4, **far), 10),
        ]
        for i, call in enumerate(calls):
            with pytest.raises(ValueError, match="different devices: cuda:[01] and cuda:[01]"):
                call()
                pytest.fail("call %d was not refused" % i)


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Named:
    """An object that names a stream, as any library may have them."""

    def __init__(self, handle):
        self.cuda_stream = handle


def test_the_check_takes_any_object_that_names_a_stream(dg):
    status = dg.det_gemm_check(Named(0))
    assert isinstance(status, int)
    assert (status == 0) == torch.cuda.is_available()


def test_the_check_needs_no_native_binding(dg):
    code = ("import sys; sys.modules['invariant_deterministic_gemm_gb300._ops_native'] = None\n"
            "import invariant_deterministic_gemm_gb300 as dg\n"
            "class Named: cuda_stream = 0\n"
            "assert isinstance(dg.det_gemm_check(Named()), int)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_operators_run_on_any_object_that_names_a_stream(dg):
    side = torch.cuda.Stream()
    x = torch.randn(100, 16, device="cuda")
    want = dg.det_moe_route(x, 2)
    torch.cuda.synchronize()
    got = dg.det_moe_route(x, 2, stream=Named(side.cuda_stream))
    assert dg.det_gemm_check(Named(side.cuda_stream)) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_an_argument_without_a_truth_value_is_refused(dg):
    both = torch.tensor([True, False])
    with pytest.raises(RuntimeError, match="ambiguous"):
        dg.det_ops_debug_force_timeout(both)
    with pytest.raises(RuntimeError, match="ambiguous"):
        dg.det_fp8_quantize_tiles(torch.zeros(16, 16, dtype=torch.bfloat16), transposed=both)


@pytest.mark.gpu
def test_what_the_library_refuses_is_not_allocated_first(dg):
    x = torch.zeros(4096, 64, device="cuda")
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for call in (lambda: dg.det_moe_route(x, 1 << 24), lambda: dg.det_moe_route(x, 33), lambda: dg.det_moe_route(x, -3),
                 lambda: dg.det_moe_dispatch(ids, 1 << 40), lambda: dg.det_moe_dispatch(ids, 513), lambda: dg.det_moe_dispatch(ids, -9)):
        with pytest.raises(dg.DetGemmError, match="INVALID_ARG"):
            call()
    assert torch.cuda.max_memory_allocated() - before < 4 << 20
