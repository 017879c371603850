"""The failure path of every GEMM, on a GPU, without a fault: as
test_gpu_timeout.py has it for LLM.int8, for the other kinds. The forward that
runs out of time returns with QLIN_ERR_TIMEOUT in the status word; the same
forward afterwards has the bits it had before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _forwards(q, M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    X = torch.randn((M, K), generator=g).to(torch.bfloat16).cuda()
    W = (0.02 * torch.randn((N, K), generator=g)).to(torch.bfloat16).cuda()
    quant = lambda mode: q.qlin_quantize_weight(W, mode)   # noqa: E731
    channel, int4, block, nvfp4 = quant(q.QLIN_W_FP8_CHANNEL), quant(q.QLIN_W_INT4_G128), quant(q.QLIN_W_INT8_BLOCK32), quant(q.QLIN_W_NVFP4)
    return {"fp8": lambda: q.qlin_fp8_forward(X, *channel, q.QLIN_W_FP8_CHANNEL), "f16": lambda: q.qlin_fp_linear_forward(X, W),
            "w4a8": lambda: q.qlin_w4a8_forward(X, *int4), "fp8_weight_only": lambda: q.qlin_fp8_weight_only_forward(X, *channel),
            "int8_block": lambda: q.qlin_int8_block_forward(X, *block), "nvfp4": lambda: q.qlin_nvfp4_weight_only_forward(X, *nvfp4)}


# K of fewer stages than any ring holds, and of more; several tiles a CTA
@pytest.mark.parametrize("M,N,K", [(300, 520, 128), (300, 520, 2048), (4200, 2056, 256)])
@pytest.mark.parametrize("kind", ["fp8", "f16", "w4a8", "fp8_weight_only", "int8_block", "nvfp4"])
def test_gemm_runs_out_of_time_and_recovers(kind, M, N, K):
    import quantized_w8a8_linear_b200 as q
    torch.cuda.init()
    assert q.qlin_get_device_status(reset=True) == q.QLIN_OK
    forward = _forwards(q, M, N, K)[kind]
    want = forward()
    assert torch.isfinite(want).all() and q.qlin_get_device_status() == q.QLIN_OK
    q.qlin_set_wait_timeout_ns(1_000_000)          # 1 ms
    q.qlin_debug_inject_wait_timeout(True)
    try:
        forward()
        status = q.qlin_get_device_status(reset=True)   # synchronises: the kernel returned
    finally:
        q.qlin_debug_inject_wait_timeout(False)
        q.qlin_set_wait_timeout_ns(2_000_000_000)
    assert status == q.QLIN_ERR_TIMEOUT
    torch.cuda.synchronize()                       # no sticky CUDA error
    assert torch.equal(forward(), want)
    assert q.qlin_get_device_status() == q.QLIN_OK
