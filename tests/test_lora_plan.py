"""What the adapters' backward asks of its caller: the partial weight gradients of
many short segments do not outgrow what they are summed to."""
import pytest

from tests.test_abi import L  # noqa: F401  (fixture: builds the library if it is missing)


@pytest.mark.parametrize("n_seg", [64, 65])
@pytest.mark.parametrize("T,K,N,R,n", [(4096, 11008, 11008, 64, 1), (4096, 4096, 4096, 128, 4), (1024, 11008, 11008, 64, 4)])
def test_workspace_of_many_segments_of_few_adapters(L, T, K, N, R, n, n_seg):  # noqa: F811
    """Sorted by adapter there is a partial sum for a block of 2 R tokens and one more for an adapter, in fp32; then
    dV with its slices, and 1 MB of the rest. One more segment does not change that."""
    tiles = -(-T // (2 * R)) + n + 1
    bound = 4 * (tiles * (K + N) * R + (-(-N // 256) + 1) * T * R) + (1 << 20)
    assert L.lib.int8_lora_backward_workspace_bytes(T, K, N, R, n, n_seg) <= bound
