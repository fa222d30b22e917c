"""Calls of the operators around a paged cache that differ from the usual ones in what surrounds them (CPU)."""
import pytest
import torch

import draft_selection_position_amd as dfs

from .test_target_pass_oracle import L  # noqa: F401


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
