"""Pins of the verification pass's oracle, and the refusals of its entry points (CPU)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import draft_selection_position_amd as dfs
from oracle import target_pass as tp

P = 0x10000  # a fake, 256-byte-aligned device address; never dereferenced by these calls
FAR = 1 << 46  # another, far from it
OK, E_NULL, E_SHAPE, E_UNSUP, E_WS, E_ALIGN, E_HIP, E_ARCH, E_ARG, E_TOO_LARGE = range(10)


def passes(f, *args, **kw):
    """Whether a call gets past every check; made only where no device could then run it on the fake addresses."""
    return torch.cuda.device_count() > 0 or f(*args, **kw) in (E_HIP, E_ARCH)



@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dfs.lib_path()):
        pytest.skip("libdfs.so not built")
    return dfs.lib()


# ---------------------------------------------------------------- pins


def test_e4m3_codes_equal_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(tp.e4m3_decode(codes.numpy()), codes.view(torch.float8_e4m3fn).double().numpy())


def test_e4m3_rounding_equals_torchs():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 5000), rng.normal(0, 0.02, 5000), tp.E4M3, -tp.E4M3,
                        (tp.E4M3[1:] + tp.E4M3[:-1]) / 2]).astype(np.float32)
    np.testing.assert_array_equal(tp.e4m3_round(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_norm_pins():
    y, scale, v, s = tp.norm_q8(np.full((1, 256), 3.0), np.ones(256), eps=0.0)
    np.testing.assert_allclose(y, 1.0, rtol=1e-15)
    np.testing.assert_allclose(scale, 1 / 448, rtol=1e-15)
    np.testing.assert_allclose(v, 448.0, rtol=1e-15)
    x = np.random.default_rng(2).normal(size=(3, 200))
    t = torch.nn.functional.rms_norm(torch.from_numpy(x + 1), (200,), eps=1e-5).numpy()
    np.testing.assert_allclose(tp.norm_q8(x, np.ones(200), np.ones((3, 200)), 1e-5)[0], t, rtol=1e-12)
    assert tp.norm_q8(x, np.ones(200))[1].shape == (2, 3)  # the last group is short


def test_linear_pins():
    rng = np.random.default_rng(3)
    a, w = rng.normal(size=(4, 200)), rng.normal(size=(130, 200))
    one, _ = tp.linear_q8(a, np.ones((2, 4)), w, np.ones((2, 2)))
    np.testing.assert_allclose(one, a @ w.T, rtol=1e-12)
    sa, sw = rng.uniform(1, 2, (2, 4)), rng.uniform(1, 2, (2, 2))
    full = (a * np.repeat(sa, 128, 0)[:200].T) @ (w * np.repeat(np.repeat(sw, 128, 0)[:130], 128, 1)[:, :200]).T
    np.testing.assert_allclose(tp.linear_q8(a, sa, w, sw)[0], full, rtol=1e-12)


def test_tree_attention_pins():
    assert tp.ancestors([-1, 0, 0, 2, -2, 4, 3, 9]) == [[0], [1, 0], [2, 0], [3, 2, 0], None, [5], [6, 3, 2, 0], None]
    rng = np.random.default_rng(4)
    B, T, Hq, Hkv, D, page, n = 1, 5, 4, 2, 8, 4, 7
    q, kn, vn = rng.normal(size=(B, T, Hq, D)), rng.normal(size=(B, T, Hkv, D)), rng.normal(size=(B, T, Hkv, D))
    kp, vp = rng.normal(size=(3, Hkv, page, D)), rng.normal(size=(3, Hkv, page, D))
    table = np.array([[2, 0, -1]])
    out = tp.tree_attention(q, kn, vn, [[-1, 0, 1, 2, 3]], kp, vp, table, [n], 0.3)[0]
    # a chain is causal attention over the concatenated sequence
    k = np.concatenate([np.concatenate([kp[2], kp[0]], 1)[:, :n], kn[0].transpose(1, 0, 2)], 1)
    v = np.concatenate([np.concatenate([vp[2], vp[0]], 1)[:, :n], vn[0].transpose(1, 0, 2)], 1)
    mask = torch.ones(T, n + T, dtype=torch.bool).tril(n)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[0].transpose(1, 0, 2)), torch.from_numpy(k).repeat_interleave(2, 0),
        torch.from_numpy(v).repeat_interleave(2, 0), attn_mask=mask, scale=0.3)
    np.testing.assert_allclose(out[0].transpose(1, 0, 2), want.numpy(), rtol=1e-10)


def test_commit_pins():
    kn = np.arange(2 * 3 * 1 * 2).reshape(2, 3, 1, 2)
    kp = np.zeros((4, 1, 2, 2), int)
    k, v, lens = tp.cache_commit(kn, kn + 100, np.array([[2, 0], [1, 2]]), [2, 5], kp, kp, np.array([[3, 1], [0, 9]]), [1, 1])
    assert lens.tolist() == [3, 3]
    assert k[3, 0, 1].tolist() == kn[0, 2, 0].tolist() and k[1, 0, 0].tolist() == kn[0, 0, 0].tolist()
    assert v[0, 0, 1].tolist() == (kn[1, 1, 0] + 100).tolist()  # the second one's page is not one of the pool's
    assert (k != 0).any(axis=-1).sum() == 3


# ---------------------------------------------------------------- refusals


def test_norm_q8_refusals(L):
    def f(x=P, r=P + (1 << 32), w=P + (2 << 32), dt=1, rows=4, d=256, eps=1e-6, q=FAR, s=FAR + (1 << 32), t=FAR + (2 << 32), y=FAR + (3 << 32)):
        return L.dfs_norm_q8(x, r, w, dt, rows, d, eps, q, s, t, y, None)

    for name in ("x", "w", "q", "s"):
        assert f(**{name: None}) == E_NULL
    assert f(dt=2) == E_UNSUP and f(d=24) == E_UNSUP
    assert f(rows=0) == E_SHAPE and f(rows=(1 << 22) + 1) == E_SHAPE and f(d=0) == E_SHAPE and f(d=65552) == E_SHAPE
    assert f(rows=1 << 22, d=16384) == E_SHAPE
    for name in ("x", "r", "w", "q", "t", "y"):
        assert f(**{name: FAR + (9 << 32) + 8}) == E_ALIGN
    assert f(s=FAR + 2) == E_ALIGN
    assert f(eps=-1.0) == E_ARG and f(eps=float("nan")) == E_ARG
    assert f(r=None) == E_ARG  # a sum without a residual
    assert f(q=P) == E_ARG and f(y=P) == E_ARG and f(t=P + 16) == E_ARG and f(t=FAR + 64) == E_ARG
    assert f(t=P + (2 << 32)) == E_ARG  # the weight's place
    assert passes(f) and passes(f, t=P) and passes(f, t=P + (1 << 32)) and passes(f, r=None, t=None, y=None)


def test_linear_q8_refusals(L):
    def f(a=P, sa=P + (1 << 32), w=P + (2 << 32), sw=P + (3 << 32), rows=4, N=100, K=256, dt=1, out=FAR, ws=FAR + (1 << 40), wsb=1 << 34):
        return L.dfs_linear_q8(a, sa, w, sw, rows, N, K, dt, out, ws, wsb, None)

    for name in ("a", "sa", "w", "sw", "out"):
        assert f(**{name: None}) == E_NULL
    assert f(dt=3) == E_UNSUP and f(K=40) == E_UNSUP
    assert f(rows=0) == E_SHAPE and f(N=0) == E_SHAPE and f(K=0) == E_SHAPE and f(K=(1 << 20) + 16) == E_SHAPE
    assert f(rows=1 << 22, N=1 << 14) == E_SHAPE and L.dfs_linear_q8_workspace_bytes(1 << 22, 1 << 14, 256) == 0
    for name in ("a", "w", "out"):
        assert f(**{name: FAR + 8}) == E_ALIGN
    assert f(sa=P + 2) == E_ALIGN and f(sw=P + 2) == E_ALIGN and f(ws=FAR + 64) == E_ALIGN
    assert f(out=P) == E_ARG and f(out=P + (3 << 32)) == E_ARG
    need = L.dfs_linear_q8_workspace_bytes(1, 5120, 4096)
    if need:
        assert f(rows=1, N=5120, K=4096, ws=None) == E_WS and f(rows=1, N=5120, K=4096, wsb=need - 1) == E_WS
    assert passes(f)


def _shape(**kw):
    v = dict(batch=2, T=5, q_heads=8, kv_heads=2, head_dim=64, page_size=16, n_pages=100, table_width=8, dtype=1) | kw
    return dfs._CacheShape(*v.values())


BAD_SHAPES = [(dict(batch=0), E_SHAPE), (dict(batch=65537), E_SHAPE), (dict(T=0), E_SHAPE), (dict(T=65), E_SHAPE),
              (dict(kv_heads=0), E_SHAPE), (dict(batch=65536, kv_heads=128, q_heads=128), E_SHAPE),
              (dict(page_size=0), E_SHAPE), (dict(page_size=24), E_UNSUP), (dict(page_size=1 << 17), E_SHAPE),
              (dict(n_pages=0), E_SHAPE), (dict(table_width=0), E_SHAPE), (dict(table_width=1 << 27), E_SHAPE),
              (dict(dtype=9), E_UNSUP), (dict(head_dim=12), E_UNSUP), (dict(head_dim=0), E_SHAPE)]


def test_tree_attention_refusals(L):
    names = ["q", "kn", "vn", "par", "kp", "vp", "tab", "lens"]

    def f(shape=None, scale=0.1, out=FAR, ws=FAR + (1 << 40), wsb=1 << 36, null=None, **ptr):
        s = _shape(**(shape or {}))
        args = [None if n == null else ptr.get(n, P + (i << 36)) for i, n in enumerate(names)]
        return L.dfs_tree_attention(*args, ctypes.byref(s), scale, out, ws, wsb, None)

    for n in names:
        assert f(null=n) == E_NULL
    assert f(out=None) == E_NULL
    for kw, code in BAD_SHAPES + [(dict(q_heads=9), E_UNSUP), (dict(q_heads=0), E_SHAPE), (dict(q_heads=1026), E_SHAPE),
                                  (dict(head_dim=96), E_UNSUP), (dict(dtype=0), E_UNSUP)]:
        assert f(kw) == code, kw
        assert L.dfs_tree_attention_workspace_bytes(ctypes.byref(_shape(**kw))) == 0
    for n in names:
        assert f(**{n: FAR + (9 << 36) + 2}) == E_ALIGN
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert f(scale=scale) == E_ARG
    for i in range(len(names)):
        assert f(out=P + (i << 36)) == E_ARG
    assert L.dfs_tree_attention_workspace_bytes(ctypes.byref(_shape())) == 0  # few cached keys at most: nothing is cut
    long = dict(table_width=400)
    need = L.dfs_tree_attention_workspace_bytes(ctypes.byref(_shape(**long)))
    assert need > 0 and f(long, ws=None) == E_WS and f(long, wsb=need - 1) == E_WS
    assert f(ws=FAR + (1 << 40) + 8) == E_ALIGN and f(long, ws=FAR + (1 << 40) + 8) == E_ALIGN
    assert passes(f) and passes(f, shape=long)


def test_cache_commit_refusals(L):
    names = ["kn", "vn", "nodes", "counts", "kp", "vp", "tab", "lens"]

    def f(shape=None, path=3, out=FAR, null=None, **ptr):
        s = _shape(**(shape or {}))
        a = [None if n == null else ptr.get(n, P + (i << 36)) for i, n in enumerate(names)]
        return L.dfs_cache_commit(*a[:4], path, *a[4:], ctypes.byref(s), out, None)

    for n in names:
        assert passes(f, null=n) if n == "nodes" else f(null=n) == E_NULL
    for kw, code in BAD_SHAPES:
        assert f(kw) == code, kw
    assert f(path=0) == E_SHAPE and f(path=6) == E_SHAPE
    for n in names:
        assert f(**{n: FAR + (9 << 36) + 2}) == E_ALIGN
    assert f(out=FAR + 2) == E_ALIGN
    for i in range(len(names)):
        assert f(out=P + (i << 36)) == E_ARG
    assert f(kp=P) == E_ARG and f(vp=P + (4 << 36)) == E_ARG  # a pool over the new keys; the two pools the same
    assert passes(f) and passes(f, out=None) and passes(f, dict(dtype=0, head_dim=8))


def test_binding_refusals():
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.norm_q8(x, torch.ones(256))
    with pytest.raises(ValueError, match="HIP device"):
        dfs.linear_q8(x, x, x, x)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.tree_attention(x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.cache_commit(x, x, None, x, x, x, x, x)
