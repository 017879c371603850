"""The failure path of the adapters' tile kernels, on a GPU, without a fault:
the test switch makes each MMA warp wait on a barrier that nothing arrives on,
so the wait runs out after a short limit. Every kernel must return with
QLIN_ERR_TIMEOUT in the device status word (copies drained, TMEM freed,
cluster barriers reached), and the calls that follow must be right."""
import pytest
import torch

from tests.test_gpu_lora import _case, _check_forward, _forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_w8a8_linear_b200 as q
    torch.cuda.init()
    assert q.qlin_get_device_status(reset=True) == 0
    yield q
    assert q.qlin_get_device_status() == 0


def _timed_out(q, call):
    q.qlin_set_wait_timeout_ns(1_000_000)          # 1 ms
    q.qlin_debug_inject_wait_timeout(True)
    try:
        call()
        status = q.qlin_get_device_status(reset=True)   # synchronises: the kernels returned
    finally:
        q.qlin_debug_inject_wait_timeout(False)
        q.qlin_set_wait_timeout_ns(2_000_000_000)
    torch.cuda.synchronize()                       # no sticky CUDA error
    assert status == q.QLIN_ERR_TIMEOUT
    assert q.qlin_get_device_status() == q.QLIN_OK


# one CTA a tile, fewer stages than the ring and more; clusters; ranks above 64; rows of odd widths
@pytest.mark.parametrize("M,K,N,L,R,idx", [(9700, 144, 64, 3, 16, "spans"), (9700, 1040, 72, 3, 16, "spans"), (300, 1040, 200, 2, 16, "tokens"),
                                           (300, 4096, 129, 4, 120, "tokens")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward_runs_out_of_time_and_recovers(q, M, K, N, L, R, idx, dtype):
    c = _case(M, K, N, L, R, dtype, idx, 30)
    _timed_out(q, lambda: _forward(q, c))
    c = _case(300, 528, 63, 4, R, dtype, "tokens", 31)
    H = torch.full((300, R), 77.0, device="cuda")
    Y, _, _ = _forward(q, c, H)
    _check_forward(c, Y, H, dtype)


@pytest.mark.parametrize("M,K,N,L,R,idx", [(300, 1040, 200, 3, 16, "tokens"), (3000, 416, 680, 3, 32, "tokens"), (1300, 528, 272, 3, 128, "spans")])
def test_backward_runs_out_of_time_and_recovers(q, M, K, N, L, R, idx):
    c = _case(M, K, N, L, R, torch.bfloat16, idx, 32)
    H = torch.zeros((M, R), device="cuda")
    _, plan, d = _forward(q, c, H)
    run = lambda: q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], plan, H, dX=d["dX"].clone())   # noqa: E731
    want = run()
    _timed_out(q, run)
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
