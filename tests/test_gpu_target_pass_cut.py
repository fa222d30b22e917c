"""Tree attention where the keys of all sequences are cut over the workgroups, on the GPU against the oracle: more
sequences than a wave has lanes, pieces that are not finite, every place of the last keys, one long sequence
among short ones.  A table for more keys than the sequences have makes their keys cut whatever the lengths are;
each test says that it does (scratch memory is for joining cut sequences, and asked for by nothing else)."""
import pytest
import torch

from oracle import target_pass as tp

from .test_gpu_target_pass import check_attention, dfs, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make_cut(dfs, seed, lens, T, Hkv, group, D, page, kind="chain", fill=None, capacity=4096):
    """test_gpu_target_pass.make with a table for `capacity` positions, entries past a sequence's pages far outside."""
    a = make(seed, lens, T, Hkv, group, D, page, kind, fill)
    width = max(a[6].shape[1], capacity // page)
    table = torch.full((len(lens), width), -(1 << 30), dtype=torch.int32, device="cuda")
    table[:, :a[6].shape[1]] = a[6]
    a[6] = table
    assert dfs.tree_attention_workspace_bytes(len(lens), T, Hkv * group, Hkv, D, page, a[4].shape[0], width) > 0
    return a


# Rows of a head by nodes and heads of a group: up to 32, to 64, to 96, to 128, more
ROWS = [(2, 2), (9, 5), (23, 4), (16, 8), (33, 4)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("batch", [3, 16, 65, 193])
def test_many_sequences(dfs, D, T, group, batch):
    if batch == 193 and T * group > 45:
        batch = 70
    lens = [(37 * b + 11) % 150 for b in range(batch)]
    lens[batch // 2] = 1300 if T * group < 64 else 700
    lens[batch - 1] = 0
    check_attention(dfs, *make_cut(dfs, batch + T, lens, T, 1, group, D, 16, "random"))


def test_six_hundred_sequences(dfs):
    lens = [(53 * b) % 70 for b in range(600)]
    lens[311], lens[599] = 2500, 900
    check_attention(dfs, *make_cut(dfs, 5, lens, 2, 2, 2, 64, 16, "chain"))
    check_attention(dfs, *make_cut(dfs, 6, lens, 1, 1, 40, 128, 64, "chain"))


def test_sequences_with_nothing_cached(dfs):
    check_attention(dfs, *make_cut(dfs, 7, [0] * 100, 5, 1, 2, 128, 32, "holes"))
    check_attention(dfs, *make_cut(dfs, 8, [0] * 100, 17, 1, 4, 64, 32, "holes"))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group", [(5, 2), (20, 3), (33, 4)])
def test_ignores_what_is_not_seen(dfs, D, T, group):
    """NaN and infinities in the pages' other rows, in unused nodes and in nodes of other branches."""
    for bad in (float("nan"), float("inf"), -float("inf")):
        a = make_cut(dfs, 7, [70, 0, 129, 400], T, 2, group, D, 16, "holes")
        b = make_cut(dfs, 7, [70, 0, 129, 400], T, 2, group, D, 16, "holes", fill=bad)
        want = dfs.tree_attention(*a)
        sees = [tp.ancestors(p) for p in a[3].tolist()]
        kill = torch.tensor([[s is None for s in q] for q in sees], device="cuda")
        leaf = [next(t for t in reversed(range(T)) if sees[i][t] is not None) for i in range(4)]
        hit = torch.zeros(4, T, dtype=torch.bool, device="cuda")
        for i, n in enumerate(leaf):
            hit[i, n] = True
        for t in (1, 2):
            b[t][kill | hit] = bad
        got = dfs.tree_attention(*b)
        assert torch.equal(got[~hit].view(torch.int16), want[~hit].view(torch.int16))
        assert not torch.isfinite(got[hit].float()).any()
        assert (got[kill] == 0).all()


def put(a, pool, pos, value, col=None):
    """value at a position of sequence 0's cached keys (pool 4) or values (5)."""
    page = a[4].shape[2]
    row = a[pool][int(a[6][0, pos // page]), :, pos % page]
    row[:, slice(None) if col is None else col] = value


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group", [(1, 4), (5, 2), (20, 3), (33, 4)])
def test_pieces_that_are_not_finite(dfs, D, T, group):
    """Infinite values in the first piece, in the last, in both with opposite signs, in a node; a NaN key and a NaN
    query; the other columns, rows and sequences as without them."""
    def args():
        return make_cut(dfs, 31, [1000, 300], T, 2, group, D, 16, "chain")

    clean = dfs.tree_attention(*args())
    a = args()
    inf = float("inf")
    put(a, 5, 3, inf, 5)
    put(a, 5, 990, -inf, 6)
    put(a, 5, 4, inf, 7)
    put(a, 5, 991, -inf, 7)
    put(a, 5, 500, float("nan"), 8)
    a[2][0, T - 1, 0, 9] = -inf
    got = dfs.tree_attention(*a)
    out = got[0].float()
    assert (out[..., 5] == inf).all() and (out[..., 6] == -inf).all() and torch.isnan(out[..., 7:9]).all()
    assert (out[T - 1, :group, 9] == -inf).all()
    for x in (got, clean):
        x[0, :, :, 5:9] = 0
        x[0, T - 1, :group, 9] = 0
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))

    clean = dfs.tree_attention(*args())
    a = args()
    put(a, 4, 640, float("nan"), 11)
    got = dfs.tree_attention(*a)
    assert torch.isnan(got[0].float()).all()
    assert torch.equal(got[1].view(torch.int16), clean[1].view(torch.int16))
    a = args()
    a[0][0, T - 1, 1] = float("nan")
    got = dfs.tree_attention(*a)
    assert torch.isnan(got[0, T - 1, 1].float()).all()
    got[0, T - 1, 1] = clean[0, T - 1, 1]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group,page", [(3, 2, 8), (16, 4, 64), (17, 4, 16), (64, 2, 128)])
def test_nodes_behind_the_last_keys(dfs, D, T, group, page):
    """Every place that a sequence's last keys and its nodes can take in a tile and at a part's border; what lies
    behind a cache's last position (NaN here) is not read into anything."""
    for lens in (list(range(130)) + [191, 192, 193], list(range(40, 170, 3))):
        check_attention(dfs, *make_cut(dfs, 9, lens, T, 1, group, D, page, "holes", fill=float("nan")))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group", [(1, 8), (17, 4), (64, 4)])
def test_one_long_sequence_among_short_ones(dfs, D, T, group):
    """It owns nearly all parts, more than a join's lanes take in one round."""
    lens = [3] * 40
    lens[17] = 9000 if T == 1 else 6000
    check_attention(dfs, *make_cut(dfs, 12, lens, T, 1, group, D, 64, "random", capacity=32768))
    check_attention(dfs, *make_cut(dfs, 13, lens[17:19], T, 1, group, D, 64, "random", capacity=32768))


def test_a_wide_table_gives_the_same_rows(dfs):
    """Whole sequences in a short table and cut ones in a wide one: within both tolerances of each other, and each
    the same bits every time."""
    a = make(14, [61, 5, 40], 33, 2, 1, 64, 16, "random")
    b = make_cut(dfs, 14, [61, 5, 40], 33, 2, 1, 64, 16, "random")
    check_attention(dfs, *a)
    first = dfs.tree_attention(*b)
    check_attention(dfs, *b, got=first)
    for _ in range(3):
        assert torch.equal(dfs.tree_attention(*b).view(torch.int16), first.view(torch.int16))
