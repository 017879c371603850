"""Scratch sizes of the layer norm's and the adapters' backward passes, exactly
(CPU only): a size that is larger than needed would pass a bound unnoticed."""
import pytest

from tests.test_abi import q  # noqa: F401  (the built library)


@pytest.mark.parametrize("K,most", [(16, 296), (1024, 296), (1040, 592), (2560, 592), (4096, 296), (16384, 296)])
def test_layer_norm_backward_workspace(q, K, most):
    # two rows of K fp32 column sums for each CTA, at most one CTA a row
    for M in (1, 7, most - 1, most, most + 1, 1 << 20):
        assert q.qlin_workspace_bytes(q.QLIN_OP_LAYER_NORM_BACKWARD, M, 0, K) == 8 * K * min(M, most)


@pytest.mark.parametrize("M,R", [(1, 8), (5, 24), (512, 16), (8191, 64), (100, 128)])
def test_lora_backward_workspace(q, M, R):
    # dH in fp32, three 16-bit parts of dH and of H, and two slots of 256 columns of partial sums for 160 CTAs
    up = lambda n: (n + 255) // 256 * 256   # noqa: E731
    assert q.lib.qlin_lora_backward_workspace_bytes(M, R) == up(4 * M * R) + 2 * up(6 * M * R) + 4 * R * 2 * 256 * 160
    assert q.lib.qlin_lora_backward_workspace_bytes(-1, R) == 0 and q.lib.qlin_lora_backward_workspace_bytes(M, 0) == 0
