"""Appends whose starts break the contract, and what they may write at most."""
import pytest
import torch

from .test_gpu_paged_cache import BF16
from .test_gpu_target_pass import cache, dfs, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def guarded(t):
    """t's values amid a larger buffer, with what lies in front and behind."""
    n, guard = t.numel(), 1 << 16
    buf = torch.full((n + 2 * guard,), 9.0, dtype=t.dtype, device="cuda")
    mine = buf[guard:guard + n].view(t.shape)
    mine.copy_(t)
    return mine, (buf[:guard], buf[guard + n:])


def bits(t):
    return t.contiguous().view(torch.int16)


STARTS = {
    "any": lambda g, B: torch.randint(-5, 100, (B + 1,), generator=g, device="cuda", dtype=torch.int32),
    "falling": lambda g, B: torch.randint(-5, 100, (B + 1,), generator=g, device="cuda", dtype=torch.int32).sort(descending=True).values,
    "lowest": lambda g, B: torch.full((B + 1,), -2 ** 31, dtype=torch.int32, device="cuda"),
    "highest": lambda g, B: torch.full((B + 1,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"),
    "to and fro": lambda g, B: torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda").repeat(B // 2 + 1)[:B + 1],
    "from before": lambda g, B: torch.arange(-70, -70 + 2 * (B + 1), 2, dtype=torch.int32, device="cuda"),
    "past the rows": lambda g, B: torch.arange(0, 3 * (B + 1), 3, dtype=torch.int32, device="cuda"),
}


@pytest.mark.parametrize("kind", STARTS)
@pytest.mark.parametrize("B,room,cached", [(200, 8, 8), (200, 24, 5), (3, 24, 5), (64, 9, 2), (5000, 4, 1)])
def test_starts_that_are_not_in_order(dfs, kind, B, room, cached):
    """Whatever the starts are: nothing but rows of k and v at positions behind a sequence's own, on pages of its own, and rows of
    q turned (here by nothing) or left; nothing in front of the buffers or behind them."""
    g = gen(12 + B)
    rows, Hkv, D, page = 50, 2, 64, 4
    kp, vp, table, _ = cache(g, [room] * B, Hkv, D, page)
    lens = torch.full((B,), cached, dtype=torch.int32, device="cuda")
    x = randn(g, rows, 3 + 2 * Hkv, D, dtype=BF16)
    q, k, v = x[:, :3], x[:, 3:3 + Hkv], x[:, 3 + Hkv:]
    pools = [guarded(t) for t in (kp, vp)]
    out, out_guard = guarded(torch.full((rows, 3, D), 7.0, device="cuda", dtype=BF16))
    # what may be written: [pages, rows of a page]
    open_ = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    at = torch.arange(cached, table.shape[1] * page, device="cuda")
    pages = table[:, at // page].long()
    there = pages >= 0
    open_[pages[there], (at % page).expand(B, -1)[there]] = True
    starts = STARTS[kind](g, B)
    _, new = dfs.cache_append(q, k, v, starts, None, pools[0][0], pools[1][0], table, lens, q_out=out)
    assert ((new >= cached) & (new <= cached + rows)).all()
    for (got, guards), was, given in zip(pools, (kp, vp), (k, v)):
        assert all((s == 9.0).all() for s in guards)
        rows_of = lambda t: bits(t.transpose(1, 2)).reshape(t.shape[0] * page, Hkv * D)  # noqa: E731
        changed = (rows_of(got) != rows_of(was)).any(dim=1)
        assert not (changed & ~open_.flatten()).any()
        new_rows, all_given = rows_of(got)[changed], bits(given).reshape(rows, Hkv * D)
        if len(new_rows):
            assert (new_rows[:, None] == all_given[None]).all(dim=2).any(dim=1).all()
    assert all((s == 9.0).all() for s in out_guard)
    mine = (bits(out) == bits(q)).flatten(1).all(dim=1)
    assert (out[~mine] == 7.0).all()
