"""The verification pass's operators with arguments at the ends of their ranges, on the GPU against the oracle."""
import pytest
import torch

from .test_gpu_target_pass import check_attention, dfs, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("T,group", [(3, 2), (20, 4)])
def test_the_smallest_and_the_largest_scale(dfs, T, group):
    """Scores that vanish, or zeros times the largest factor: every key that a row sees has the same weight, and
    none that it does not see has any."""
    a = make(3, [70, 0, 129], T, 2, group, 64, 16, "holes")
    check_attention(dfs, *a, scale=2.0 ** -149)
    check_attention(dfs, *a, scale=1e-39)
    a[0].zero_()
    check_attention(dfs, *a, scale=2.3e38)
    for scale in (1e-46, 2.4e38):
        with pytest.raises(dfs.DfsError):
            dfs.tree_attention(*a, scale=scale)
