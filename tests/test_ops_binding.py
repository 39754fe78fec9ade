"""The native binding's checks that need no GPU: tensors that claim to lie on
one (PyTorch's fake tensors) are refused before their memory is asked for."""
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
