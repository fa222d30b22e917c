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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_smallest_and_the_largest_eps(dfs, dtype):
    """A row of zeros stays zero with the smallest positive eps, and any row is zero under the largest."""
    x, w = torch.zeros(3, 256, device="cuda", dtype=dtype), torch.ones(256, device="cuda", dtype=dtype)
    x[1] = 1.0
    for eps in (2.0 ** -149, 1e-39, 3.4e38):
        q, scale, y = dfs.norm_q8(x, w, eps=eps, normed=True)
        want = 1.0 if eps < 1 else (1.0 + eps) ** -0.5
        rel = torch.finfo(dtype).eps / 2 + 50 * 2.0 ** -24  # the output's rounding, the norm's own
        assert (q[[0, 2]].float() == 0).all() and (scale[:, [0, 2]] == 2.0 ** -100).all()
        assert ((y[1].double() - want).abs() <= rel * want).all()
    for eps in (1e-46, 3.5e38):
        with pytest.raises(dfs.DfsError):
            dfs.norm_q8(x, w, eps=eps)
