"""Arguments of the verification pass's operators at the ends of their ranges, and the package's import (CPU)."""
import ctypes
import subprocess
import sys

from .test_target_pass_oracle import E_ARG, FAR, L, P, _shape, passes  # noqa: F401

FP32_MAX, FP32_TINY = 3.4028234663852886e38, 2.0 ** -149


def test_a_scale_outside_fp32_is_refused(L):  # noqa: F811
    """The kernel multiplies scores by fp32(scale * log2(e)): neither zero nor infinite."""
    def f(scale):
        a = [P + (i << 36) for i in range(8)]
        return L.dfs_tree_attention(*a, ctypes.byref(_shape()), scale, FAR, FAR + (1 << 40), 1 << 36, None)

    for scale in (1e-300, 1e-46, FP32_TINY / 4, FP32_MAX, 2.4e38, 1e300):
        assert f(scale) == E_ARG, scale
    for scale in (FP32_TINY, 1e-30, 1.0, 2.3e38):
        assert passes(f, scale), scale


def test_an_eps_outside_fp32_is_refused(L):  # noqa: F811
    """The kernel adds fp32(eps): a positive one may not become zero, nor a finite one infinite."""
    def f(eps):
        return L.dfs_norm_q8(P, None, P + (2 << 32), 1, 4, 256, eps, FAR, FAR + (1 << 32), None, None, None)

    for eps in (1e-300, FP32_TINY / 4, 3.5e38, 1e300):
        assert f(eps) == E_ARG, eps
    for eps in (0.0, FP32_TINY, 1e-6, FP32_MAX):
        assert passes(f, eps), eps


def test_imports_where_torch_has_no_gpu_streams():
    """As in a CPU build of torch, which lacks the call that gives a device's current stream."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import draft_selection_position_amd as dfs\n"
            "x = torch.zeros(2, 256)\n"
            "try:\n    dfs.norm_q8(x, x[0])\nexcept ValueError as e:\n    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "HIP device" in r.stdout
