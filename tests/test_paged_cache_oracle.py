"""Pins of the oracle of the operators around a paged cache, the frequencies' schedules (host code), and the entry
points' refusals (CPU)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import draft_selection_position_amd as dfs
from oracle import paged_cache as pc
from oracle import target_pass as tp

from .test_target_pass_oracle import BAD_SHAPES, E_ALIGN, E_ARG, E_NULL, E_SHAPE, E_UNSUP, E_WS, FAR, OK, P, _shape, passes


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dfs.lib_path()):
        pytest.skip("libdfs.so not built")
    return dfs.lib()


# ---------------------------------------------------------------- pins


def test_positions_pins():
    got = pc.tree_positions([[-1, 0, 1, 2], [-1, 0, -2, 2], [5, -1, 1, 0]], [10, 0, -3], 7)
    assert got.tolist() == [[17, 18, 19, 20], [7, 8, 7, 7], [7, 7, 8, 7]]
    assert pc.tree_positions([[-1, 0]], [2 ** 31 - 1], 2 ** 31 - 1).tolist() == [[2 ** 31 - 1] * 2]


def test_rotation_pins():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2, 8))
    f = np.array([1.0, 0.1, 0.01])
    assert np.array_equal(pc.rotate(x, [0, 0, 0], f)[0], x)
    for layout, one, two in (("half", [0, 1, 2], [3, 4, 5]), ("interleaved", [0, 2, 4], [1, 3, 5])):
        y, _ = pc.rotate(x, [5, 7, 11], f, layout)
        z = (x[..., one] + 1j * x[..., two]) * np.exp(1j * np.outer([5, 7, 11], f))[:, None]
        np.testing.assert_allclose(y[..., one] + 1j * y[..., two], z, rtol=1e-13)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        np.testing.assert_allclose(pc.rotate(y, [-5, -7, -11], f, layout)[0], x, rtol=1e-12)  # back again
        # a turned query's product with a turned key depends on the distance alone
        a, b = pc.rotate(x, [40, 40, 40], f, layout)[0], pc.rotate(x, [43, 43, 43], f, layout)[0]
        c, d = pc.rotate(x, [0, 0, 0], f, layout)[0], pc.rotate(x, [3, 3, 3], f, layout)[0]
        np.testing.assert_allclose((a[0] * b[1]).sum(-1), (c[0] * d[1]).sum(-1), rtol=1e-10)
    np.testing.assert_allclose(pc.rotate(x, [5, 7, 11], f, "half", 1.5)[0][..., :6], 1.5 * pc.rotate(x, [5, 7, 11], f)[0][..., :6])


def test_slots_pins():
    table = np.array([[3, 1], [0, 9]])
    got = pc.append_slots([1, 3, 6], 7, table, [1, 2], 4, 2, prefix=10)
    assert got == [None, (11, 3, 1), (12, 1, 0), (12, None, 0), (13, None, 1), (14, None, 0), None]


def test_shared_attention_pins():
    """A prefix in a table of its own is the same as the prefix's pages in front of every sequence's."""
    rng = np.random.default_rng(4)
    B, T, Hq, Hkv, D, page = 2, 3, 4, 2, 8, 4
    q, kn, vn = rng.normal(size=(B, T, Hq, D)), rng.normal(size=(B, T, Hkv, D)), rng.normal(size=(B, T, Hkv, D))
    kp, vp = rng.normal(size=(9, Hkv, page, D)), rng.normal(size=(9, Hkv, page, D))
    par = [[-1, 0, 0], [-1, -2, 0]]
    own, pre = np.array([[2, 0], [5, 6]]), np.array([8, 3])
    a = pc.tree_attention_shared(q, kn, vn, par, kp, vp, pre, 8, own, [5, 0], 0.3)
    b = tp.tree_attention(q, kn, vn, par, kp, vp, np.concatenate([np.tile(pre, (2, 1)), own], axis=1), [13, 8], 0.3)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-12)
    a = pc.tree_attention_shared(q, kn, vn, par, kp, vp, pre, 0, own, [5, 0], 0.3)
    np.testing.assert_allclose(a[0], tp.tree_attention(q, kn, vn, par, kp, vp, own, [5, 0], 0.3)[0], rtol=1e-12)


# ---------------------------------------------------------------- frequencies (host)


@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128, 1024])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, original=4096.0),
                                dict(scaling="yarn", factor=1.0, original=4096.0),
                                dict(scaling="yarn", factor=4.0, original=100.0, beta_fast=3.0, beta_slow=2.9),
                                dict(scaling="bands", factor=8.0, original=8192.0, beta_fast=4.0, beta_slow=1.0)])
def test_frequencies(L, rot, base, kw):
    if kw.get("scaling") == "ntk" and rot == 2:
        with pytest.raises(dfs.DfsError):
            dfs.rope_frequencies(rot, base, **kw)
        return
    f, a = dfs.rope_frequencies(rot, base, **kw)
    want, amplitude = pc.frequencies(rot, base, **kw)
    assert f.dtype == torch.float32 and f.shape == (rot // 2,)
    # a rounding to fp32, and some of 64 bits
    np.testing.assert_allclose(f.double().numpy(), want, rtol=2.0 ** -24 + 1e-12, atol=2.0 ** -150)
    assert abs(a - amplitude) <= 1e-15
    if not kw:
        assert a == 1.0 and f[0] == 1.0


def test_frequencies_ends():
    """What each schedule does to the fastest and the slowest pairs."""
    plain = pc.frequencies(128, 10000.0)[0]
    for scaling in ("yarn", "bands"):
        f, _ = dfs.rope_frequencies(128, 10000.0, scaling, 8.0, 4096.0, 32.0, 1.0)
        assert f[0] == 1.0 and abs(f[-1].item() * 8 / plain[-1] - 1) < 1e-6 and (f.diff() < 0).all()
    f, _ = dfs.rope_frequencies(128, 10000.0, "ntk", 8.0)
    assert f[0] == 1.0 and abs(f[-1].item() * 8 / plain[-1] - 1) < 1e-6


def test_frequencies_refusals(L):
    out = (ctypes.c_float * 512)()

    def f(rot=64, base=1e4, scaling=3, factor=4.0, original=4096.0, fast=32.0, slow=1.0, to=out):
        return L.dfs_rope_frequencies(rot, base, scaling, factor, original, fast, slow, to, None)

    assert f() == OK and f(scaling=0, factor=float("nan"), original=-1.0) == OK and f(scaling=1, original=0.0) == OK
    assert f(to=None) == E_NULL
    assert f(rot=0) == E_SHAPE and f(rot=1026) == E_SHAPE and f(rot=7) == E_UNSUP
    assert f(scaling=5) == E_UNSUP and f(scaling=-1) == E_UNSUP
    nan, inf = float("nan"), float("inf")
    for kw in (dict(base=1.0), dict(base=nan), dict(base=inf), dict(factor=0.5), dict(factor=nan), dict(factor=inf),
               dict(original=0.0), dict(original=nan), dict(original=inf), dict(fast=1.0), dict(slow=0.0), dict(fast=nan),
               dict(slow=nan), dict(fast=inf)):
        assert f(**kw) == E_ARG, kw
    with pytest.raises(ValueError, match="scaling"):
        dfs.rope_frequencies(64, scaling="cubic")
    for rot in (0, -2, 3):
        with pytest.raises(dfs.DfsError):
            dfs.rope_frequencies(rot)


# ---------------------------------------------------------------- refusals


def test_tree_positions_refusals(L):
    def f(par=P, lens=P + (1 << 32), pre=P + (2 << 32), batch=4, T=5, out=FAR):
        return L.dfs_tree_positions(par, lens, pre, batch, T, out, None)

    for n in ("par", "lens", "out"):
        assert f(**{n: None}) == E_NULL
        assert f(**{n: FAR + (9 << 32) + 2}) == E_ALIGN
    assert f(pre=P + 2) == E_ALIGN
    for kw in (dict(batch=0), dict(batch=65537), dict(T=0), dict(T=65), dict(batch=-1), dict(batch=1 << 62)):
        assert f(**kw) == E_SHAPE
    for out in (P, P + 76, P + (1 << 32) + 12, P + (2 << 32)):
        assert f(out=out) == E_ARG
    assert passes(f) and passes(f, pre=None) and passes(f, out=P + 80) and passes(f, batch=65536, T=64)


def _rope(**kw):
    v = dict(rows=10, q_heads=8, kv_heads=2, head_dim=64, rot_dim=64, q_stride=768, k_stride=768, v_stride=768,
             amplitude=1.0, layout=0, dtype=1) | kw
    return dfs._RopeShape(*v.values())


BAD_ROPES = [(dict(rows=0), E_SHAPE), (dict(rows=(1 << 22) + 1), E_SHAPE), (dict(kv_heads=0), E_SHAPE), (dict(q_heads=0), E_SHAPE),
             (dict(kv_heads=1025), E_SHAPE), (dict(q_heads=1025), E_SHAPE), (dict(head_dim=0), E_SHAPE), (dict(head_dim=1032), E_SHAPE),
             (dict(head_dim=68), E_UNSUP), (dict(rot_dim=66), E_SHAPE), (dict(rot_dim=-2), E_SHAPE), (dict(rot_dim=63), E_UNSUP),
             (dict(q_stride=504), E_SHAPE), (dict(k_stride=120), E_SHAPE), (dict(v_stride=0), E_SHAPE), (dict(q_stride=1 << 32), E_SHAPE),
             (dict(k_stride=(1 << 62) + 8), E_SHAPE), (dict(v_stride=772), E_UNSUP), (dict(layout=2), E_UNSUP), (dict(layout=-1), E_UNSUP),
             (dict(dtype=2), E_UNSUP), (dict(amplitude=0.0), E_ARG), (dict(amplitude=-1.0), E_ARG), (dict(amplitude=float("nan")), E_ARG),
             (dict(amplitude=float("inf")), E_ARG), (dict(amplitude=1e-60), E_ARG), (dict(amplitude=1e60), E_ARG)]


def test_rope_refusals(L):
    names = ["q", "k", "v", "pos", "freqs"]
    outs = ["oq", "ok", "ov"]

    def f(shape=None, null=(), **ptr):
        s = _rope(**(shape or {}))
        a = [None if n in null else ptr.get(n, P + (i << 36)) for i, n in enumerate(names)]
        o = [None if n in null else ptr.get(n, FAR + (i << 36)) for i, n in enumerate(outs)]
        return L.dfs_rope(*a, ctypes.byref(s), *o, None)

    for n in names + outs:
        assert f(null=(n,)) == E_NULL  # an input without its output, or the other way round, too
    assert f(null=("q", "oq", "k", "ok")) == E_NULL
    assert L.dfs_rope(P, P, P, P, P, None, FAR, FAR, FAR, None) == E_NULL
    for kw, code in BAD_ROPES + [(dict(rot_dim=0), E_SHAPE)]:
        assert f(kw) == code, kw
    for n in names + outs:
        assert f(**{n: FAR + (9 << 36) + 2}) == E_ALIGN
        if n not in ("pos", "freqs"):
            assert f(**{n: FAR + (9 << 36) + 8}) == E_ALIGN
    for i in range(len(names)):
        for o in outs:
            assert f(**{o: P + (i << 36)}) == E_ARG
    assert f(ok=FAR) == E_ARG and f(ov=FAR + (1 << 36) + 2544) == E_ARG  # two outputs
    dense = dict(q_stride=512, k_stride=128, v_stride=128)
    assert passes(f, dense, oq=P, ok=P + (1 << 36))  # in place
    assert f(dense, ov=P + (2 << 36)) == E_ARG and f(dense, oq=P + 16) == E_ARG
    assert passes(f) and passes(f, null=("v", "ov")) and passes(f, null=("k", "ok", "v", "ov")) and passes(f, null=("q", "oq"))
    assert passes(f, dict(kv_heads=0, k_stride=0, v_stride=0), null=("k", "ok", "v", "ov"))
    assert passes(f, dict(q_heads=0, q_stride=0), null=("q", "oq")) and passes(f, dict(rot_dim=2, layout=1, dtype=0))


def test_cache_append_refusals(L):
    names = ["q", "k", "v", "starts", "freqs", "pre", "kp", "vp", "tab", "lens"]

    def f(rope=None, shape=None, null=(), oq=FAR, ol=FAR + (1 << 40), **ptr):
        r, s = _rope(**(rope or {})), _shape(**(shape or {}))
        a = {n: None if n in null else ptr.get(n, P + (i << 36)) for i, n in enumerate(names)}
        if "oq" in null:
            oq = None
        return L.dfs_cache_append(a["q"], a["k"], a["v"], a["starts"], a["freqs"], ctypes.byref(r), a["pre"], oq, a["kp"],
                                  a["vp"], a["tab"], a["lens"], ctypes.byref(s), ol, None)

    for n in names + ["oq"]:
        assert passes(f, null=(n,)) if n == "pre" else f(null=(n,)) == E_NULL, n
    assert L.dfs_cache_append(None, P, P, P, P, None, None, None, P, P, P, P, ctypes.byref(_shape()), None, None) == E_NULL
    assert L.dfs_cache_append(None, P, P, P, P, ctypes.byref(_rope()), None, None, P, P, P, P, None, None, None) == E_NULL
    for kw, code in BAD_ROPES:
        assert f(kw) == code, kw
    for kw, code in BAD_SHAPES:
        assert (passes(f, None, kw) if "T" in kw else f(None, kw) == code), kw
    for kw in (dict(kv_heads=4), dict(head_dim=128), dict(dtype=0)):
        assert f(None, kw) == E_SHAPE
    for n in names:
        assert f(**{n: FAR + (9 << 36) + 2}) == E_ALIGN
    assert f(ol=FAR + (1 << 40) + 2) == E_ALIGN and f(oq=FAR + 8) == E_ALIGN
    for i in range(len(names)):
        assert f(ol=P + (i << 36)) == E_ARG and f(oq=P + (i << 36)) == E_ARG
    for n in ("kp", "vp"):
        for i in (0, 1, 2, 3, 4, 5, 8, 9):
            assert f(**{n: P + (i << 36)}) == E_ARG
    assert f(vp=P + (6 << 36) + 1024) == E_ARG  # the two pools
    assert passes(f) and passes(f, ol=None) and passes(f, null=("q", "oq")) and passes(f, dict(rot_dim=0), null=("freqs",))
    assert passes(f, dict(q_stride=512), oq=P)  # the query in place


def test_shared_attention_refusals(L):
    names = ["q", "kn", "vn", "par", "kp", "vp", "ptab", "plen", "tab", "lens"]

    def f(shape=None, width=50, scale=0.1, out=FAR, ws=FAR + (1 << 40), wsb=1 << 38, null=None, **ptr):
        s = _shape(**(shape or {}))
        a = [None if n == null else ptr.get(n, P + (i << 36)) for i, n in enumerate(names)]
        return L.dfs_tree_attention_shared(*a[:8], width, *a[8:], ctypes.byref(s), scale, out, ws, wsb, None)

    need = lambda width=50, **kw: L.dfs_tree_attention_shared_workspace_bytes(ctypes.byref(_shape(**kw)), width)  # noqa: E731
    for n in names:
        assert f(null=n) == E_NULL
    assert f(out=None) == E_NULL
    for kw, code in BAD_SHAPES + [(dict(q_heads=9), E_UNSUP), (dict(q_heads=0), E_SHAPE), (dict(q_heads=1026), E_SHAPE),
                                  (dict(head_dim=96), E_UNSUP), (dict(dtype=0), E_UNSUP)]:
        assert f(kw) == code, kw
        assert need(**kw) == 0
    for width in (0, -1, (1 << 26) + 1, 1 << 62):
        assert f(width=width) == E_SHAPE and need(width) == 0
    for n in names:
        assert f(**{n: FAR + (9 << 36) + 2}) == E_ALIGN
    for scale in (0.0, -1.0, float("inf"), float("nan"), 1e-46, 1e39):
        assert f(scale=scale) == E_ARG
    for i in range(len(names)):
        assert f(out=P + (i << 36)) == E_ARG
    n = need()
    assert n > 0 and f(ws=None) == E_WS and f(wsb=n - 1) == E_WS and f(ws=FAR + (1 << 40) + 8) == E_ALIGN
    assert passes(f) and passes(f, wsb=n) and passes(f, width=1 << 26)


def test_plans_over_extreme_sizes(L):
    """The workspace query for any sizes: no crash, no overflow; 2^45 bytes are more than any call in range needs."""
    for batch in (-1, 0, 1, 3, 64, 65536, 1 << 62):
        for T in (0, 1, 17, 64, 65):
            for kv, q in ((1, 1), (1, 1024), (8, 32), (1024, 1024), (1 << 40, 1 << 40)):
                for page, table in ((1, 1), (16, 100), (65536, 16384), (1 << 30, 1)):
                    for width in (-5, 1, 1000, 1 << 30):
                        s = _shape(batch=batch, T=T, q_heads=q, kv_heads=kv, head_dim=128, page_size=page, table_width=table)
                        assert L.dfs_tree_attention_shared_workspace_bytes(ctypes.byref(s), width) < 1 << 45


def test_binding_refusals():
    x, i = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32)
    f = torch.ones(32)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.tree_positions(torch.zeros(2, 3, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.rope(x, x, None, i, f)
    with pytest.raises(ValueError, match="q or k"):
        dfs.rope(None, None, x, i, f)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        dfs.rope(x.half(), None, None, i, f)
    with pytest.raises(TypeError):
        dfs.rope([1], None, None, i, f)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.cache_append(None, x, x, i, f, x, x, i, i)
    with pytest.raises(TypeError):
        dfs.cache_append(None, x, None, i, f, x, x, i, i)
    with pytest.raises(ValueError, match="HIP device"):
        dfs.tree_attention_shared(x, x, x, x, x, x, x, x, x, x)
