"""Attention over a shared prefix where lengths, pages, scores and streams are out of the ordinary, by each way that few rows
take: few keys in one launch; the prefix by tree attention's kernel with the own keys in the same launch; and with these in a
launch of their own, either of which leaves pieces.  (The prefix's own kernel: test_gpu_shared_prefix.py.)

The way goes by the tables' widths.  That a call takes the way it is meant for shows in the scratch memory that it needs: the
first takes none but the least.
"""
import pytest
import torch

from .test_gpu_paged_cache import BF16, check_rotated, frequencies, i32, make_shared
from .test_gpu_paged_cache_use import Pools, bits
from .test_gpu_shared_prefix import ancestors_mask, check, wide
from .test_gpu_target_pass import dfs, gen, randn, trees  # noqa: F401

pytestmark = pytest.mark.gpu
WAYS = ["one launch", "beside", "apart"]
LEAST = 256  # bytes of scratch


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def scratch(dfs, a):  # noqa: F811
    B, T, Hq, D = a[0].shape
    n, Hkv, page = a[4].shape[:3]
    return dfs.tree_attention_shared_workspace_bytes(B, T, Hq, Hkv, D, page, n, a[8].shape[1], a[6].shape[0])


def by(dfs, way, a):  # noqa: F811
    """The same call with tables as wide as `way` needs."""
    page = a[4].shape[2]
    a = list(a)
    if way != "one launch":
        before = scratch(dfs, a)
        a[6] = wide(a[6], 2000 // page + 1)
        beside = scratch(dfs, a)
        assert beside > LEAST and before != beside
        if way == "apart":
            a[8] = wide(a[8], 9000 // page + 1)
            assert scratch(dfs, a) not in (LEAST, beside)
    else:
        assert scratch(dfs, a) == LEAST
    return a


def clamped(a):
    """The tables as the library reads them, for the dense computation."""
    n = a[4].shape[0]
    return [*a[:6], a[6].clamp(0, n - 1), i32([min(max(int(a[7]), 0), a[6].shape[0] * a[4].shape[2])]), a[8].clamp(0, n - 1), a[9]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way", WAYS)
def test_lengths_out_of_range(dfs, way, D):
    """A prefix's length beyond its table, or below zero; pages that the pool does not have, in either table."""
    a = by(dfs, way, make_shared(25, 64, [20, 5], 3, 1, 2, D, 16))
    most = a[6].shape[0] * 16
    if way == "one launch":
        a[6], most = a[6][:4].contiguous(), 64
        assert scratch(dfs, a) == LEAST
    full = [*a[:7], i32([most]), *a[8:]]
    want = dfs.tree_attention_shared(*full)
    check(dfs, clamped(full), got=want)
    for n in (2 ** 31 - 1, most + 1):
        a[7] = i32([n])
        assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(want))
    none = dfs.tree_attention_shared(*a[:7], i32([0]), *a[8:])
    check(dfs, [*a[:7], i32([0]), *a[8:]], got=none)
    for n in (-3, -2 ** 31):
        a[7] = i32([n])
        assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(none))
    a[7] = i32([64])
    n = a[4].shape[0]
    a[6][:4] = i32([2 ** 31 - 1, -5, n, 0])
    a[8][0, :2] = i32([-2 ** 31, n])
    got = dfs.tree_attention_shared(*a)
    assert torch.equal(bits(got), bits(dfs.tree_attention_shared(*clamped(a))))
    check(dfs, clamped(a), got=got)


@pytest.mark.parametrize("way", WAYS)
def test_own_lengths_out_of_range(dfs, way):
    a = by(dfs, way, make_shared(26, 40, [32, 5, 0], 4, 2, 1, 64, 16, "random"))
    a[9] = i32([32, -7, -2 ** 31])
    want = dfs.tree_attention_shared(*a[:9], i32([32, 0, 0]))
    assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(want))
    check(dfs, [*a[:9], i32([32, 0, 0])], got=want)
    most = a[8].shape[1] * 16
    a[9] = i32([2 ** 31 - 1, 5, most + 3])
    want = dfs.tree_attention_shared(*a[:9], i32([most, 5, most]))
    assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(want))
    check(dfs, clamped([*a[:9], i32([most, 5, most])]), got=want)


@pytest.mark.parametrize("way", WAYS)
def test_infinite_scores(dfs, way):
    """A key whose scores are all -inf weighs nothing; rows that see nothing else are zero."""
    a = by(dfs, way, make_shared(24, 20, [0, 0], 1, 1, 1, 64, 4))
    a[0].fill_(1.0)
    a[1].fill_(-float("inf"))  # the nodes' own keys
    out = dfs.tree_attention_shared(*a)
    a[3][:] = -1
    kp, vp, ptab = a[4], a[5], a[6]
    pos = torch.arange(20, device="cuda")
    k, v = (p[ptab[pos // 4].long(), 0, pos % 4].double() for p in (kp, vp))
    w = torch.softmax(a[0][0, 0].double() @ k.t().contiguous() / 8, dim=1)
    # weights and output rounded to bf16, 2^-8 each of the weighted |v| at most, and less than that of fp32
    assert (out[:, 0].double() - (w @ v)).abs().max() <= 3 * 2.0 ** -8 * v.abs().max()
    a[7] = i32([0])
    assert (dfs.tree_attention_shared(*a) == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("big", ["prefix", "own"])
def test_scores_far_apart(dfs, big, way, D):
    """Weights of the prefix, or of the sequence's own keys, that vanish beside the other's."""
    a = by(dfs, way, make_shared(22, 150, [90, 30], 4, 1, 2, D, 16, qstd=1.0))
    q, kp, ptab, table = a[0], a[4], a[6], a[8]
    q.fill_(1.0)
    pages = ptab[:10].long() if big == "prefix" else table[:, :6].clamp(min=0).unique().long()
    kp[pages] = kp[pages] * 0.1 + 12.0
    check(dfs, a)


@pytest.mark.parametrize("way", WAYS)
def test_unused_nodes(dfs, way):
    """A tree of unused nodes only: zeros, whatever its queries hold; the others as they were."""
    a = by(dfs, way, make_shared(21, 300, [40, 7, 0], 12, 2, 2, 64, 16))
    clean = dfs.tree_attention_shared(*a)
    a[3][1] = -2
    a[0][1] = float("nan")
    out = dfs.tree_attention_shared(*a)
    assert (out[1] == 0).all()
    assert torch.equal(bits(out[0]), bits(clean[0])) and torch.equal(bits(out[2]), bits(clean[2]))
    a[0][1] = 0
    check(dfs, a, got=out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_what_no_sequence_owns_is_not_read(dfs, fill, way, D):
    for prefix, lens, T, page in ((37, [5, 0], 3, 16), (0, [9, 9], 2, 8), (100, [64, 1], 9, 64), (64, [0, 64], 1, 1)):
        check(dfs, by(dfs, way, make_shared(prefix, prefix, lens, T, 1, 2, D, page, "random", fill=fill)))


@pytest.mark.parametrize("way", WAYS)
def test_not_finite_where_it_is_seen(dfs, way):
    """A NaN in a query stays in its row, one in a node's value in the rows that see the node, one in the prefix reaches all that are used."""
    a = by(dfs, way, make_shared(27, 100, [33, 0, 50], 6, 1, 2, 64, 16, "holes"))
    want = dfs.tree_attention_shared(*a)
    tree = ancestors_mask(a[3])
    used = tree.any(dim=2)
    b, t = used.nonzero()[2].tolist()
    a[0][b, t] = float("nan")
    got = dfs.tree_attention_shared(*a)
    assert torch.isnan(got[b, t].float()).all()
    got[b, t] = want[b, t]
    assert torch.equal(bits(got), bits(want))
    a[0][b, t] = 0.5
    want = dfs.tree_attention_shared(*a)
    a[2][b, t, 0, 7] = float("nan")
    got, sees = dfs.tree_attention_shared(*a), tree[b, :, t]
    assert torch.isnan(got[b, sees][..., 7].float()).all() and torch.equal(bits(got[b, ~sees]), bits(want[b, ~sees]))
    a[2][b, t, 0, 7] = 0.5
    a[5][a[6][2].long(), 0, 3, 11] = float("nan")
    got = dfs.tree_attention_shared(*a)
    assert torch.isnan(got[used][..., 11].float()).all() and torch.isfinite(got[used][..., :11].float()).all()
    assert (got[~used] == 0).all()


@pytest.mark.parametrize("ways", [("beside", "apart"), ("one launch", "beside"), ("apart", "apart")])
def test_two_streams_at_once(dfs, ways):
    """Each with pieces of its own."""
    calls = [by(dfs, ways[0], make_shared(50, 300, [90, 10], 5, 2, 4, 64, 16)), by(dfs, ways[1], make_shared(51, 200, [20, 300], 14, 2, 1, 128, 16))]
    want = [dfs.tree_attention_shared(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(dfs.tree_attention_shared(*calls[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for t in got[i]:
            assert torch.equal(bits(t), bits(want[i]))


@pytest.mark.parametrize("way", WAYS)
def test_captured_and_replayed(dfs, way):
    """Two graphs of a step each (append and attention), replayed with eager work and synchronisation between, on changed inputs, own
    lengths and prefix lengths."""
    g = gen(61)
    B, T, Hq, Hkv, D, page = 3, 4, 8, 2, 64, 16
    pool = Pools(g, Hkv, D, page, 9, B, 4)
    f = frequencies(D)
    lens, plen, starts = i32([0, 5, 10]), i32([133]), i32(list(range(B + 1)))
    par = trees(g, B, T, "random")
    inputs = [(randn(g, B, T, Hq, D, dtype=BF16), randn(g, B, T, Hkv, D, dtype=BF16), randn(g, B, T, Hkv, D, dtype=BF16),
               randn(g, B, 2 * Hkv, D, dtype=BF16)) for _ in range(4)]
    a = by(dfs, way, [inputs[0][0], inputs[0][1], inputs[0][2], par, pool.k, pool.v, pool.prefix, plen, pool.table, lens])
    ptab, table = a[6], a[8]

    def work(q, k, v, y):
        _, new = dfs.cache_append(None, y[:, :Hkv], y[:, Hkv:], starts, f, pool.k, pool.v, table, lens, prefix_len=plen)
        return [dfs.tree_attention_shared(q, k, v, par, pool.k, pool.v, ptab, plen, table, new), new]

    static = [[t.clone() for t in inputs[i]] for i in range(2)]
    work(*static[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in static:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work(*x))
        graphs.append(graph)
    for turn in range(6):
        for i in range(2):
            for t, s in zip(static[i], inputs[(turn + i) % 4]):
                t.copy_(s)
            plen.fill_([133, 0, 64, 144, 1, 2 ** 31 - 1][turn])
            lens.copy_(i32([[0, 5, 10], [50, 0, 3], [15, 16, 17]][turn % 3]))
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            mine = [t.clone() for t in outs[i]] + [pool.k.clone(), pool.v.clone()]
            eager = work(*static[i]) + [pool.k, pool.v]  # the same append again
            for x, y in zip(mine, eager):
                assert torch.equal(bits(x), bits(y)), (turn, i)
            if turn != 5:
                check(dfs, [*static[i][:3], par, pool.k, pool.v, ptab, plen, table, eager[1]], got=mine[0])


@pytest.mark.parametrize("way", WAYS)
def test_one_workspace_for_calls_in_turn(dfs, way):
    """What an earlier call of another size left in it, or nothing but ones, changes nothing."""
    calls = [by(dfs, way, make_shared(73, 200, [60, 0, 90], 5, 2, 4, 64, 16)), by(dfs, way, make_shared(74, 90, [20, 7], 9, 3, 1, 128, 16))]
    ws = torch.full((max(scratch(dfs, a) for a in calls),), 255, dtype=torch.uint8, device="cuda")
    want = [dfs.tree_attention_shared(*a) for a in calls]
    for i in (0, 1, 1, 0, 0, 1):
        assert torch.equal(bits(dfs.tree_attention_shared(*calls[i], workspace=ws)), bits(want[i]))
    ws.fill_(255)
    for i in (1, 0):
        assert torch.equal(bits(dfs.tree_attention_shared(*calls[i], workspace=ws)), bits(want[i]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way", WAYS)
def test_a_pool_past_32_bits(dfs, way, D):
    """The prefix's pages and the sequences' behind 2^32 bytes of the pools."""
    g = gen(81)
    Hkv, page = 8, 64
    n = 40000 * 128 // D  # 5.2 GB a pool
    kp, vp = (torch.zeros((n, Hkv, page, D), dtype=BF16, device="cuda") for _ in range(2))
    table = i32([[n - 1, n - 1000, 0], [n - 2, n - 1001, 1]])
    prefix = i32([n - 3, n - 2000, n - 3000])
    f = frequencies(D)
    x = randn(g, 330, 2 * Hkv, D, dtype=BF16)
    _, plen = dfs.cache_append(None, x[:150, :Hkv], x[:150, Hkv:], i32([0, 150]), f, kp, vp, prefix[None], i32([0]))
    _, lens = dfs.cache_append(None, x[150:, :Hkv], x[150:, Hkv:], i32([0, 100, 180]), f, kp, vp, table, i32([0, 0]), prefix_len=plen)
    check_rotated(kp[n - 2000, :, 3:5].transpose(0, 1), x[67:69, :Hkv], [67, 68], f, "half", 1.0)
    B, T = 2, 3
    q, k, v = (randn(g, B, T, Hkv, D, dtype=BF16) for _ in range(3))
    par = trees(g, B, T, "chain")
    a = by(dfs, way, [q, k, v, par, kp, vp, prefix, plen, table, lens])
    out = dfs.tree_attention_shared(*a)
    used = sorted({*table.flatten().tolist(), *prefix.tolist()})
    small = lambda t: i32([[used.index(p) for p in row] for row in t.tolist()])  # noqa: E731
    check(dfs, [q, k, v, par, kp[used], vp[used], small(prefix[None])[0], plen, small(table), lens], got=out)
