"""The operators around a paged cache as they are used: a prompt and its sequences into the cache, a pass over drafted
trees, the accepted nodes, the next pass; captured and replayed, on other streams, with offsets past 32 bits, and
refusals by the binding."""
import numpy as np
import pytest
import torch

from oracle import paged_cache as pc

from .test_gpu_paged_cache import BF16, check_rotated, check_shared, frequencies, i32, make_shared
from .test_gpu_shared_prefix import check, large
from .test_gpu_target_pass import dfs, gen, randn, trees  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.uint8)


class Pools:
    """A pool with tables of its own for a prefix and for B sequences."""

    def __init__(self, g, Hkv, D, page, prefix_pages, B, pages):
        n = prefix_pages + B * pages + 2
        order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.k, self.v = (randn(g, n, Hkv, page, D, dtype=BF16) for _ in range(2))
        self.prefix = order[:prefix_pages].contiguous()
        self.table = order[prefix_pages:prefix_pages + B * pages].view(B, pages).contiguous()


def test_a_shared_prompt_and_its_answers(dfs):
    """A prompt into the cache once, each sequence's own beginning behind it, a pass over drafted trees, the accepted path into
    the cache, and a pass of single tokens: every step against the oracle on what it was given."""
    g = gen(1)
    B, T, Hq, Hkv, D, page, P = 3, 6, 8, 2, 64, 16, 75
    freqs, amplitude = dfs.rope_frequencies(D, 10000.0, "yarn", 4.0, 4096.0, device="cuda")
    pool = Pools(g, Hkv, D, page, 5, B, 6)
    heads = lambda t: (t[..., :Hq, :], t[..., Hq:Hq + Hkv, :], t[..., Hq + Hkv:, :])  # noqa: E731
    # the prompt, as one sequence of a table that is the prefix's
    prompt = randn(g, P, Hq + 2 * Hkv, D, dtype=BF16)
    _, plen = dfs.cache_append(None, *heads(prompt)[1:], i32([0, P]), freqs, pool.k, pool.v, pool.prefix[None], i32([0]),
                               amplitude=amplitude)
    assert plen.tolist() == [P]
    at = torch.arange(P, device="cuda")
    cached = pool.k[pool.prefix[at // page].long(), :, at % page]
    check_rotated(cached, heads(prompt)[1], range(P), freqs, "half", amplitude)
    # ragged beginnings of the sequences
    starts = [0, 9, 9, 40]
    own = randn(g, 40, Hq + 2 * Hkv, D, dtype=BF16)
    q, lens = dfs.cache_append(*heads(own), i32(starts), freqs, pool.k, pool.v, pool.table, i32([0, 0, 0]), amplitude=amplitude,
                               prefix_len=plen)
    assert lens.tolist() == [9, 0, 31]
    pos = [P + r - starts[b] for b in range(B) for r in range(starts[b], starts[b + 1])]
    check_rotated(q, heads(own)[0], pos, freqs, "half", amplitude)
    # a pass over drafted trees: heads out of one projection's rows
    par = trees(g, B, T, "random")
    qkv = randn(g, B, T, Hq + 2 * Hkv, D, dtype=BF16)
    where = dfs.tree_positions(par, lens, plen)
    assert np.array_equal(where.cpu().numpy(), pc.tree_positions(par.tolist(), lens.tolist(), P))
    q, k, v = dfs.rope(*heads(qkv), where, freqs, amplitude=amplitude)
    for got, raw in ((q, heads(qkv)[0]), (k, heads(qkv)[1])):
        check_rotated(got.reshape(B * T, -1, D), raw.reshape(B * T, -1, D), where.flatten().tolist(), freqs, "half", amplitude)
    assert torch.equal(v, heads(qkv)[2])
    check_shared(dfs, q, k, v, par, pool.k, pool.v, pool.prefix, plen, pool.table, lens)
    # a path of accepted nodes
    chains = [seen[::-1] for seen in (pc.ancestors(row)[-1] for row in par.tolist())]
    nodes = i32([c + [0] * (T - len(c)) for c in chains])
    counts = i32([len(c) for c in chains])
    before = pool.k.clone(), pool.v.clone()
    new = dfs.cache_commit(k, v, nodes, counts, pool.k, pool.v, pool.table, lens)
    assert torch.equal(new, lens + counts)
    # the same as if the path's tokens had been appended
    rows = torch.tensor([b * T + n for b, c in enumerate(chains) for n in c], device="cuda")
    path = [t.reshape(B * T, -1, D)[rows] for t in heads(qkv)[1:]]
    cum = np.concatenate([[0], np.cumsum([len(c) for c in chains])]).tolist()
    dfs.cache_append(None, *path, i32(cum), freqs, *before, pool.table, lens, amplitude=amplitude, prefix_len=plen)
    assert torch.equal(before[0], pool.k) and torch.equal(before[1], pool.v)
    # the next pass, a token each
    par1 = trees(g, B, 1, "chain")
    qkv = randn(g, B, 1, Hq + 2 * Hkv, D, dtype=BF16)
    q, k, v = dfs.rope(*heads(qkv), dfs.tree_positions(par1, new, plen), freqs, amplitude=amplitude)
    check_shared(dfs, q, k, v, par1, pool.k, pool.v, pool.prefix, plen, pool.table, new)


def test_attention_depends_on_distances_alone(dfs):
    """Everything some tokens further on: turned queries and keys meet as before."""
    g = gen(2)
    D, n = 128, 40
    f = frequencies(D)
    q, k = randn(g, 1, 1, D), randn(g, n, 1, D)
    dots = []
    for far in (0, 1000):
        a = dfs.rope(q, None, None, i32([n + far]), f)[0]
        b = dfs.rope(None, k, None, i32(range(far, far + n)), f)[1]
        dots.append((a.double() * b.double()).sum(dim=2))
    # each value within 8 u of |x1| + |x2| of its pair (see the rotation's tolerance), which is at most sqrt(2) of its norm
    bound = 2 * 8 * 2.0 ** -24 * 1.5 * (q.double().norm() * k.double().norm(dim=2))
    assert ((dots[0] - dots[1]).abs() <= 2 * bound).all()


def test_the_same_call_gives_the_same_bits(dfs):
    for a in (make_shared(3, 700, [60, 0, 300], 17, 2, 4, 128, 16, "random"), large(make_shared(4, 900, [30] * 30, 17, 2, 1, 64, 16, "random"))):
        first = dfs.tree_attention_shared(*a)
        for _ in range(5):
            assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(first))


def test_two_streams_at_once(dfs):
    calls = [make_shared(50, 300, [90, 10], 5, 2, 4, 64, 16), large(make_shared(51, 500, [20] * 30, 14, 2, 1, 128, 16))]
    want = [dfs.tree_attention_shared(*c) for c in calls]
    qkv, f, pos = randn(gen(52), 200, 6, 64, dtype=BF16), frequencies(64), torch.arange(200, dtype=torch.int32, device="cuda")
    turned = dfs.rope(qkv[:, :4], qkv[:, 4:], None, pos, f)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append((dfs.tree_attention_shared(*calls[i]), dfs.rope(qkv[:, :4], qkv[:, 4:], None, pos, f)))
    torch.cuda.synchronize()
    for i in range(2):
        for t, r in got[i]:
            assert torch.equal(bits(t), bits(want[i])) and torch.equal(r[0], turned[0]) and torch.equal(r[1], turned[1])


@pytest.mark.parametrize("many", [False, True])
def test_captured_and_replayed(dfs, many):
    """Two graphs of a whole step each (positions, rotation, append, attention), replayed with eager work and
    synchronisation between, on changed inputs and lengths."""
    g = gen(61)
    B, T, Hq, Hkv, D, page = (40, 12, 2, 2, 64, 16) if many else (3, 4, 8, 2, 64, 16)
    pool = Pools(g, Hkv, D, page, 9, B, 4)
    ptab = pool.prefix
    if many:  # a table wide enough for the prefix's own kernel
        ptab = torch.cat([ptab, torch.full((3 * 2 ** 32 // (B * T * Hkv * D * page) + 1,), -1, dtype=torch.int32, device="cuda")])
    f = frequencies(D)
    lens, plen = i32([(5 * b) % 30 for b in range(B)]), i32([133])
    par = trees(g, B, T, "random")
    starts = i32(list(range(B + 1)))
    inputs = [(randn(g, B, T, Hq + 2 * Hkv, D, dtype=BF16), randn(g, B, 2 * Hkv, D, dtype=BF16)) for _ in range(4)]
    cut = lambda t: (t[..., :Hq, :], t[..., Hq:Hq + Hkv, :], t[..., Hq + Hkv:, :])  # noqa: E731

    def work(x, y):
        _, new = dfs.cache_append(None, y[:, :Hkv], y[:, Hkv:], starts, f, pool.k, pool.v, pool.table, lens, prefix_len=plen)
        q, k, v = dfs.rope(*cut(x), dfs.tree_positions(par, new, plen), f)
        return [dfs.tree_attention_shared(q, k, v, par, pool.k, pool.v, ptab, plen, pool.table, new), q, k, v, new]

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
            plen.fill_([133, 0, 64, 144, 1, 100][turn])
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            mine = [t.clone() for t in outs[i]] + [pool.k.clone(), pool.v.clone()]
            eager = work(*static[i]) + [pool.k, pool.v]  # the same append again
            for a, b in zip(mine, eager):
                assert torch.equal(bits(a), bits(b)), (turn, i)


def test_a_pool_past_32_bits(dfs):
    g = gen(81)
    Hkv, page, D, n = 8, 64, 128, 40000  # 5.2 GB a pool
    kp, vp = (torch.zeros((n, Hkv, page, D), dtype=BF16, device="cuda") for _ in range(2))
    table = i32([[n - 1, 39000, 0], [n - 2, 38999, 1]])
    prefix = i32([n - 3, 38000, 37000])
    f = frequencies(D)
    x = randn(g, 330, 2 * Hkv, D, dtype=BF16)
    _, plen = dfs.cache_append(None, x[:150, :Hkv], x[:150, Hkv:], i32([0, 150]), f, kp, vp, prefix[None], i32([0]))
    _, lens = dfs.cache_append(None, x[150:, :Hkv], x[150:, Hkv:], i32([0, 100, 180]), f, kp, vp, table, i32([0, 0]), prefix_len=plen)
    check_rotated(kp[38000, :, 3:5].transpose(0, 1), x[67:69, :Hkv], [67, 68], f, "half", 1.0)
    assert torch.equal(vp[n - 2, :, 9], x[259, Hkv:]) and torch.equal(vp[39000, :, 35], x[249, Hkv:])
    used = sorted({*table.flatten().tolist(), *prefix.tolist()})
    small = lambda t: i32([[used.index(p) for p in row] for row in t.tolist()])  # noqa: E731
    for B in (2, 80):
        T, reps = (3, 1) if B == 2 else (5, 40)
        q, k, v = randn(g, B, T, Hkv, D, dtype=BF16), randn(g, B, T, Hkv, D, dtype=BF16), randn(g, B, T, Hkv, D, dtype=BF16)
        a = [q, k, v, trees(g, B, T, "chain"), kp, vp, prefix, plen, table.repeat(reps, 1), lens.repeat(reps)]
        if B > 2:
            a = large(a)
        out = dfs.tree_attention_shared(*a)
        check(dfs, a[:4] + [kp[used], vp[used], small(prefix[None])[0], plen, small(table).repeat(reps, 1), lens.repeat(reps)], got=out)


def test_rows_past_32_bits(dfs):
    rows, H, D = 270000, 64, 128  # 2.2e9 values
    x = torch.randn((rows, H, D), generator=gen(83), device="cuda", dtype=BF16)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f = frequencies(D)
    pick = [0, 1, 262143, 262144, rows - 1]
    was = x[pick]
    got = dfs.rope(x, None, None, pos, f)[0]
    check_rotated(got[pick], was, pick, f, "half", 1.0)
    dfs.rope(x, None, None, pos, f, out=(x, None, None))
    for r in range(0, rows, 30000):
        assert torch.equal(x[r:r + 30000], got[r:r + 30000])


def test_strides_of_all_kinds(dfs):
    """Rows that are one of a batch, apart by more than their heads, of one head, and of a transposed batch."""
    g = gen(84)
    f = frequencies(32)
    big = randn(g, 4, 9, 5, 32)
    pos = torch.arange(36, dtype=torch.int32, device="cuda")
    for x, p in ((big[:, :, 1:3], pos.view(4, 9)), (big[:, 3:4, 4:], pos[:4].view(4, 1)), (big[1:2, :, :, :], pos[:9].view(1, 9)),
                 (big[2, ::2, :2], pos[:5])):
        got = dfs.rope(x, None, None, p.contiguous(), f)[0]
        check_rotated(got.reshape(-1, *x.shape[-2:]), x.reshape(-1, *x.shape[-2:]), p.flatten().tolist(), f, "half", 1.0)
    for bad in (big.transpose(0, 1)[:, :, :2], big[..., ::2], big.transpose(1, 2), big[:, :, :1].expand(-1, -1, 3, -1)):
        with pytest.raises(ValueError):
            dfs.rope(bad, None, None, torch.zeros(bad.shape[:-2], dtype=torch.int32, device="cuda"), f[:bad.shape[-1] // 2].contiguous())
    with pytest.raises(dfs.DfsError):  # one row for all of them
        dfs.rope(big[:, :1, :2].expand(-1, 9, -1, -1)[0], None, None, pos[:9], f)


# ---------------------------------------------------------------- the binding's refusals


def test_binding_refuses(dfs):
    g = gen(91)
    par, lens, one = trees(g, 3, 4, "chain"), i32([1, 2, 3]), i32([7])
    for bad in ((par.long(), lens), (par, lens[:2]), (par[0], lens), (par, lens.long()), (par.cpu(), lens), (par, lens, lens), (par, lens, one.long()),
                (par.t(), lens)):
        with pytest.raises(ValueError):
            dfs.tree_positions(*bad)
    with pytest.raises(TypeError):
        dfs.tree_positions(par, None)
    with pytest.raises(dfs.DfsError):
        dfs.tree_positions(par[:, :0].contiguous(), lens)
    with pytest.raises(dfs.DfsError):
        dfs.tree_positions(par, lens, out=par)
    with pytest.raises(ValueError):
        dfs.tree_positions(par, lens, out=par[:, :2].contiguous())

    q, k, v = randn(g, 5, 4, 64, dtype=BF16), randn(g, 5, 2, 64, dtype=BF16), randn(g, 5, 2, 64, dtype=BF16)
    pos, f = i32(range(5)), frequencies(64)
    for bad, kw in (((q.half(), k, v, pos, f), {}), ((q, k.float(), v, pos, f), {}), ((q, k, v[:4], pos, f), {}), ((q, k, v[:, :1], pos, f), {}),
                    ((q, k[..., :32], v, pos, f), {}), ((q, k, v, pos.long(), f), {}), ((q, k, v, pos[:4], f), {}), ((q, k, v, pos, f.double()), {}),
                    ((q, k, v, pos, f[None]), {}), ((q, k, v, pos, f), dict(layout="pairs")), ((q.cpu(), k, v, pos, f), {}), ((q, k.cpu(), v, pos, f), {}),
                    ((q, k, v, pos.cpu(), f), {}), ((q[0], None, None, pos, f), {}), ((q, k, v, pos, f), dict(out=(q, k))),
                    ((q, k, v, pos, f), dict(out=(q, k, None))), ((q, k, None, pos, f), dict(out=(q, v[:4], None)))):
        with pytest.raises(ValueError):
            dfs.rope(*bad, **kw)
    for bad in ((q, k, v, None, f), (q, k, v, pos, None), (q, [1], v, pos, f)):
        with pytest.raises(TypeError):
            dfs.rope(*bad)
    with pytest.raises(dfs.DfsError):
        dfs.rope(q, k, v, pos, f, amplitude=0.0)
    with pytest.raises(dfs.DfsError):  # more than a head has
        dfs.rope(q, k, v, pos, frequencies(66))
    with pytest.raises(dfs.DfsError):
        dfs.rope(q[:0], None, None, pos[:0], f)
    with pytest.raises(dfs.DfsError):  # v in its own place
        dfs.rope(q, k, v, pos, f, out=(q, k, v))
    with pytest.raises(dfs.DfsError):
        dfs.rope(q, k, None, pos, f, out=(k.new_empty(q.shape), q.view(-1)[:k.numel()].view(k.shape), None))  # k's over q

    kp, vp = randn(g, 9, 2, 16, 64, dtype=BF16), randn(g, 9, 2, 16, 64, dtype=BF16)
    table, st = i32([[0, 1], [2, 3]]), i32([0, 2, 5])
    good = [q, k, v, st, f, kp, vp, table, i32([0, 0])]
    for i, bad in ((0, q.float()), (0, q[:4]), (1, k.float()), (2, v[:4]), (3, st[:2]), (3, st.long()), (4, f.double()), (5, kp[:, :1].contiguous()),
                   (5, kp.float()), (6, vp[:8]), (7, table[:1]), (7, table.t()), (8, i32([0])), (8, lens.long())):
        with pytest.raises(ValueError):
            dfs.cache_append(*good[:i], bad, *good[i + 1:])
    for kw in (dict(prefix_len=i32([1, 2])), dict(q_out=q[:4]), dict(out_lens=i32([0])), dict(layout=1)):
        with pytest.raises(ValueError):
            dfs.cache_append(*good, **kw)
    with pytest.raises(ValueError):
        dfs.cache_append(None, *good[1:], q_out=q)
    for i in (1, 2, 3, 5, 6, 7, 8):
        with pytest.raises(TypeError):
            dfs.cache_append(*good[:i], None, *good[i + 1:])
    with pytest.raises(dfs.DfsError):
        dfs.cache_append(*good, out_lens=good[8])
    with pytest.raises(dfs.DfsError):
        dfs.cache_append(*good[:6], kp, *good[7:])

    a = make_shared(92, 40, [20, 3], 3, 2, 2, 64, 16)
    for i, bad in ((0, a[0].float()), (0, a[0][:, :2].contiguous()), (1, a[1].float()), (2, None), (3, a[3].long()), (3, a[3][:1]),
                   (4, a[4][:, :1].contiguous()), (6, a[6][None]), (6, a[6].long()), (6, None), (7, a[9]), (7, a[7].cpu()), (7, None), (8, a[8][:1]),
                   (9, a[9].long())):
        with pytest.raises((ValueError, TypeError)):
            dfs.tree_attention_shared(*a[:i], bad, *a[i + 1:])
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(out=a[0])):
        with pytest.raises(dfs.DfsError):
            dfs.tree_attention_shared(*a, **kw)
    with pytest.raises(ValueError):
        dfs.tree_attention_shared(*a, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        dfs.tree_attention_shared(*a, out=a[0][:1])
    with pytest.raises(dfs.DfsError):
        dfs.tree_attention_shared(*a[:6], a[6][:0].contiguous(), *a[7:])


def test_explicit_workspace_and_output(dfs):
    a = make_shared(93, 500, [50, 0], 4, 2, 2, 64, 16)
    n = dfs.tree_attention_shared_workspace_bytes(2, 4, 4, 2, 64, 16, a[4].shape[0], a[8].shape[1], a[6].shape[0])
    ws, out = torch.full((n,), 255, dtype=torch.uint8, device="cuda"), torch.empty_like(a[0])
    got = dfs.tree_attention_shared(*a, workspace=ws, out=out)
    assert got is out and torch.equal(bits(out), bits(dfs.tree_attention_shared(*a)))
