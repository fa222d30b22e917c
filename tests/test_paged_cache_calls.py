"""Calls of the operators around a paged cache that differ from the usual ones in what surrounds them (CPU)."""
import ctypes

import pytest
import torch

import draft_selection_position_amd as dfs

from .test_paged_cache_oracle import _rope
from .test_target_pass_oracle import FAR, L, P, _shape, passes  # noqa: F401


@pytest.mark.parametrize("kw", [dict(), dict(scaling="yarn", factor=8.0, original=4096.0)])
def test_frequencies_under_another_default_device(L, kw):  # noqa: F811
    """They are computed on the host, whatever device a program builds its model on."""
    want, amplitude = dfs.rope_frequencies(64, 10000.0, **kw)
    with torch.device("meta"):
        got, same = dfs.rope_frequencies(64, 10000.0, **kw)
        moved, _ = dfs.rope_frequencies(64, 10000.0, **kw, device="cpu")
        away, _ = dfs.rope_frequencies(64, 10000.0, **kw, device="meta")
    assert got.device.type == "cpu" and torch.equal(got, want) and same == amplitude
    assert torch.equal(moved, want) and away.device.type == "meta" and away.shape == want.shape


@pytest.mark.parametrize("rot", [1026, 1 << 40, 1 << 64, (1 << 64) + 64, 64 - (1 << 64), -(1 << 63), -64])
def test_frequencies_of_sizes_that_no_head_has(L, rot):  # noqa: F811
    """Refused as such, also what 64 bits do not hold, before anything is allocated or written for it."""
    with pytest.raises(dfs.DfsError, match="DFS_E_SHAPE"):
        dfs.rope_frequencies(rot)


def test_an_amplitude_is_taken_by_its_value(L, monkeypatch):  # noqa: F811
    """One that is a tensor may change between two calls of the same sizes."""
    seen = []
    tensor = lambda t, *_: isinstance(t, torch.Tensor)  # noqa: E731
    monkeypatch.setattr(dfs, "_fits", tensor)
    monkeypatch.setattr(dfs, "_on", tensor)
    monkeypatch.setattr(dfs, "_call", lambda index, where, fn, *args: seen.extend(a._obj.amplitude for a in args
                                                                                if isinstance(getattr(a, "_obj", None), dfs._RopeShape)))
    x, i, f = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32), torch.ones(32)
    pages, table, lens = torch.zeros(4, 3, 16, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    amplitude = torch.tensor(1.25)
    for value in (1.25, 2.5):
        amplitude.fill_(value)
        dfs.rope(x, None, None, i, f, amplitude=amplitude)
        dfs.cache_append(None, x, x, i, f, pages, pages.clone(), table, lens, amplitude=amplitude)
    assert seen == [1.25, 1.25, 2.5, 2.5]


@pytest.mark.parametrize("any_", [2 ** 63 - 1, -2 ** 63, 2 ** 62 + 8, -1, 0])
def test_sizes_that_are_not_looked_at(L, any_):  # noqa: F811
    """Those of heads that are not given, the rows' strides of them, and what the append does without."""
    heads = dict(q=dict(q_heads=any_, q_stride=any_), kv=dict(kv_heads=any_, k_stride=any_, v_stride=any_))

    def rope(kw, q, k, v):
        ins, outs = ([P + (i << 36) if there else None for i, there in enumerate((q, k, v))],
                     [FAR + (i << 36) if there else None for i, there in enumerate((q, k, v))])
        return L.dfs_rope(*ins, P + (4 << 36), P + (5 << 36), ctypes.byref(_rope(**kw)), *outs, None)

    assert passes(rope, heads["q"], False, True, True) and passes(rope, heads["kv"], True, False, False)
    assert passes(rope, dict(k_stride=any_), True, False, True) and passes(rope, dict(v_stride=any_), True, True, False)

    def append(rope_kw, shape_kw):
        a = [P + (i << 36) for i in range(9)]
        return L.dfs_cache_append(None, a[0], a[1], a[2], a[3], ctypes.byref(_rope(**rope_kw)), a[4], None, a[5], a[6], a[7], a[8],
                                  ctypes.byref(_shape(**shape_kw)), FAR, None)

    assert passes(append, heads["q"], dict(T=any_, q_heads=any_))
