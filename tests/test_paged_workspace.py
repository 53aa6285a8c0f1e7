"""se_paged_decode_workspace_size is 0 for every size that se_paged_decode refuses."""
import pytest


@pytest.mark.parametrize("shape,most", [((32, 4, 128, 128), 4096), ((2, 1, 64, 64), 4096), ((64, 1, 576, 512), 512)])
def test_largest_batches(se_lib, shape, most):
    f = se_lib.se_paged_decode_workspace_size
    assert f(most, *shape) == f(1, *shape) > 0
    assert f(most + 1, *shape) == 0 and f(2 ** 31 - 1, *shape) == 0
