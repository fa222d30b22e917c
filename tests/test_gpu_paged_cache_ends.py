"""The operators around a paged cache at the ends of their ranges: the most rows, heads, sequences and nodes, pages used
twice, tensors given twice, one workspace in two graphs."""
import numpy as np
import pytest
import torch

from oracle import paged_cache as pc

from .test_gpu_paged_cache import BF16, F32, SHARED, check_rotated, frequencies, i32, make_shared
from .test_gpu_shared_prefix import ancestors_mask, check, large, wide
from .test_gpu_target_pass import dfs, gen, randn, trees  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.uint8)


def test_the_most_trees(dfs):
    B, T = 65536, 64
    par = trees(gen(1), 64, T, "holes").repeat(B // 64, 1)
    lens = torch.arange(B, dtype=torch.int32, device="cuda")
    got = dfs.tree_positions(par, lens, i32([7])).view(-1, 64, T)
    depth = torch.from_numpy(pc.tree_positions(par[:64].tolist(), [0] * 64)).cuda()
    assert torch.equal(got.long(), depth + 7 + lens.view(-1, 64, 1).long())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,Hq,Hkv,D,rot", [(1 << 22, 1, 1, 8, 8), (3, 1024, 1024, 8, 2), (2, 1024, 3, 16, 16), (2, 5, 1024, 1024, 2)])
def test_rope_the_most(dfs, dtype, rows, Hq, Hkv, D, rot):
    g = gen(2)
    q, k, v = (randn(g, rows, h, D, dtype=dtype) for h in (Hq, Hkv, Hkv))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f = frequencies(rot)
    for layout in ("half", "interleaved"):
        out = dfs.rope(q, k, v, pos, f, layout=layout)
        pick = sorted({0, 1, rows // 2, rows - 1})
        for o, x in zip(out[:2], (q, k)):
            check_rotated(o[pick], x[pick], pick, f, layout, 1.0)
        assert torch.equal(out[2], v)
        # each kind alone gives the same
        assert torch.equal(dfs.rope(q, None, v, pos, f, layout=layout)[0], out[0])
        assert torch.equal(dfs.rope(None, k, None, pos, f, layout=layout)[1], out[1])


@pytest.mark.parametrize("amplitude", [1e-30, 1e30])
def test_rope_amplitudes(dfs, amplitude):
    x, pos, f = randn(gen(3), 9, 2, 64), torch.arange(9, dtype=torch.int32, device="cuda"), frequencies(32)
    check_rotated(dfs.rope(x, None, None, pos, f, amplitude=amplitude)[0], x, range(9), f, "half", amplitude)


def test_rope_of_one_tensor_as_both(dfs):
    x, pos, f = randn(gen(4), 30, 3, 64, dtype=BF16), torch.arange(30, dtype=torch.int32, device="cuda"), frequencies(64)
    q, k, v = dfs.rope(x, x, x, pos, f)
    assert torch.equal(q, k) and torch.equal(v, x)
    check_rotated(q, x, range(30), f, "half", 1.0)


@pytest.mark.parametrize("B,rows,Hkv,D,page", [(65536, 100000, 1, 8, 1), (65536, 5, 3, 16, 4), (1, 70000, 1, 8, 65536), (4096, 4096, 1024, 8, 1)])
def test_append_the_most(dfs, B, rows, Hkv, D, page):
    g = gen(B + rows)
    starts = torch.sort(torch.randint(0, rows + 1, (B + 1,), generator=g, device="cuda", dtype=torch.int32)).values
    starts[0], starts[-1] = 0, rows
    n = (starts[1:] - starts[:-1]).long()
    width = int((n.max() + page - 1) // page) + 1
    used = (n + page) // page + 1
    first = torch.cumsum(used, 0) - used
    table = (first[:, None] + torch.arange(width, device="cuda")).to(torch.int32)  # pages in a row, as far as used
    table = torch.where(torch.arange(width, device="cuda") < used[:, None], table, -1).contiguous()
    kp, vp = (torch.zeros(int(used.sum()), Hkv, page, D, dtype=BF16, device="cuda") for _ in range(2))
    lens = (torch.arange(B, device="cuda") % 2).to(torch.int32) if page > 1 else torch.zeros(B, dtype=torch.int32, device="cuda")
    x = randn(g, rows, 2 * Hkv, D, dtype=BF16)
    f = frequencies(D)
    _, new = dfs.cache_append(None, x[:, :Hkv], x[:, Hkv:], starts, f, kp, vp, table, lens)
    assert torch.equal(new.long(), lens.long() + n)
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
    at = torch.arange(rows, device="cuda") - starts.long()[b] + lens.long()[b]
    pages = table.long()[b, at // page]
    assert torch.equal(vp[pages, :, at % page], x[:, Hkv:])
    turned = dfs.rope(None, x[:, :Hkv], None, at.to(torch.int32), f)[1]
    assert torch.equal(kp[pages, :, at % page], turned)
    assert int((vp != 0).sum()) == int((x[:, Hkv:] != 0).sum())  # nothing anywhere else


@pytest.mark.parametrize("B,T,Hkv,group,D,own,width,many", [
    *((*c, many) for c in ((65536, 1, 1, 1, 64, 1, 0), (20000, 1, 1, 2, 128, 3, 3000), (1024, 64, 1, 1, 128, 2, 0),
                           (400, 1, 1024, 1, 64, 1, 0), (2, 64, 1, 64, 64, 30, 0)) for many in (False, True)),
    (1, 1, 1024, 1, 128, 5, 0, False)])
def test_shared_the_most(dfs, B, T, Hkv, group, D, own, width, many):
    """many: by the prefix's own kernel."""
    a = make_shared(B, 70, [own] * 2, T, Hkv, group, D, 16, "random")
    q = randn(gen(B), B, T, Hkv * group, D, dtype=BF16)
    rep = lambda t, n: t[torch.arange(n, device="cuda") % 2].contiguous()  # noqa: E731
    a = [q, *(rep(t, B) for t in a[1:4]), *a[4:8], wide(rep(a[8], B), width), rep(a[9], B)]
    if many:
        a = large(a)
    out = dfs.tree_attention_shared(*a)
    for lo in range(0, B, 4096):  # the dense computation by pieces
        pick = slice(lo, min(B, lo + 4096))
        check(dfs, [*(t[pick] for t in a[:4]), *a[4:8], a[8][pick], a[9][pick]], got=out[pick])


@pytest.mark.parametrize("D", [64, 128])
def test_not_finite_in_the_prefix_reaches_no_unused_node(dfs, D):
    """In one launch, by single waves, in launches of their own."""
    for lens, T, Hkv, width in (([9, 3, 40] * 4, 5, 1, 0), ([9, 3, 40] * 171, 5, 2, 0), ([9, 3, 40] * 4, 5, 1, 600), ([9] * 20, 33, 1, 0)):
        a = make_shared(71, 300, lens, T, Hkv, 1, D, 16, "holes")
        a[8] = wide(a[8], width)
        used = ancestors_mask(a[3]).any(dim=2)
        a[5][a[6][3].long(), 0, 2, 11] = float("nan")
        got = dfs.tree_attention_shared(*a)
        assert torch.isnan(got[used][:, 0, 11].float()).all() and torch.isfinite(got[used][:, 0, :11].float()).all()
        assert (got[~used] == 0).all()


def test_pages_and_tensors_given_twice(dfs):
    """A page at two places of the prefix and in a sequence's own table; keys that are the values."""
    for many in (False, True):
        a = make_shared(72, 96, [40, 20, 0] * 40, 4, 1, 1, 64, 16)
        a[6][1] = a[6][0]
        a[6][4] = a[8][0, 1]
        a[8][3, 0] = a[6][2]
        a[8][4] = a[8][0]
        a[5], a[2] = a[4], a[1]
        check(dfs, large(a) if many else a)


def test_one_workspace_in_two_graphs(dfs):
    """Nothing is kept in it from one call for the next."""
    calls = [make_shared(73, 700, [60, 0, 300], 5, 2, 4, 64, 16), large(make_shared(74, 500, [20] * 30, 14, 2, 1, 128, 16))]
    need = [dfs.tree_attention_shared_workspace_bytes(len(a[9]), a[0].shape[1], a[0].shape[2], a[4].shape[1], a[0].shape[3], 16,
                                                      a[4].shape[0], a[8].shape[1], a[6].shape[0]) for a in calls]
    ws = torch.full((max(need),), 255, dtype=torch.uint8, device="cuda")
    want = [dfs.tree_attention_shared(*a) for a in calls]
    graphs, outs = [], []
    for a in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dfs.tree_attention_shared(*a, workspace=ws))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1), (1, 0, 1)):
        for o in outs:
            o.fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(bits(o), bits(w))
        ws.fill_(order[0] * 127)


def test_prompts_in_pieces(dfs):
    """A prompt appended at once, or piece by piece, is the same cache."""
    g = gen(75)
    x, f = randn(g, 100, 6, 96, dtype=BF16), frequencies(48)
    table = torch.randperm(8, generator=g, device="cuda").to(torch.int32)[None, :7].contiguous()
    pools = [[torch.zeros(8, 2, 16, 96, dtype=BF16, device="cuda") for _ in range(2)] for _ in range(2)]
    cut = lambda t: (t[:, :2], t[:, 2:4], t[:, 4:])  # noqa: E731
    q, whole = dfs.cache_append(*cut(x), i32([0, 100]), f, *pools[0], table, i32([0]), layout="interleaved")
    lens, parts = i32([0]), []
    for lo, hi in ((0, 1), (1, 18), (18, 18 + 33), (51, 100)):
        p, lens = dfs.cache_append(*cut(x[lo:hi]), i32([0, hi - lo]), f, *pools[1], table, lens, layout="interleaved")
        parts.append(p)
    assert torch.equal(lens, whole) and torch.equal(torch.cat(parts), q)
    assert all(torch.equal(s, t) for s, t in zip(*pools))
    assert np.isfinite(q.float().cpu().numpy()).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,T,Hkv,group,page,width,many", [
    ([511, 0, 512, 513, 1023, 1024, 1025, 40], 1, 8, 4, 16, 0, False),
    ([1537, 3, 2047, 0], 5, 4, 2, 64, 0, False),
    ([2600, 0, 700, 30, 5, 1], 2, 2, 16, 1, 5000, False),               # a table for more keys than there are
    ([1500, 9, 500, 0], 4, 8, 1, 16, 0, True)])
def test_own_keys_of_many_sequences(dfs, D, lens, T, Hkv, group, page, width, many):
    n = len(lens)
    a = make_shared(76, 200, lens, T, Hkv, group, D, page, "holes")
    B = -(-1024 // Hkv)
    rep = lambda t: t[torch.arange(B, device="cuda") % n].contiguous()  # noqa: E731
    a = [randn(gen(77), B, T, Hkv * group, D, dtype=BF16), *(rep(t) for t in a[1:4]), *a[4:8], wide(rep(a[8]), width // page), rep(a[9])]
    if many:
        a = large(a)
    out = dfs.tree_attention_shared(*a)
    for lo in range(0, B, 256):
        check(dfs, [*(t[lo:lo + 256] for t in a[:4]), *a[4:8], a[8][lo:lo + 256], a[9][lo:lo + 256]], got=out[lo:lo + 256])
    assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(out))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix,lens,T,Hkv,group,page,kind", [
    (0, [0, 0], 1, 1, 1, 1, "chain"), (1, [0, 5], 1, 3, 4, 1, "chain"), (127, [0, 1, 70], 5, 2, 4, 16, "holes"),  # up to 32 rows
    (128, [200, 0], 8, 2, 4, 32, "random"), (300, [77, 31, 33], 3, 1, 8, 64, "holes"),
    (2, [65, 0, 40], 26, 3, 2, 1, "chain"), (33, [0, 31, 64], 20, 2, 3, 8, "holes"), (64, [64, 1], 64, 1, 1, 64, "random"),  # up to 64
    (97, [30, 3], 24, 1, 4, 16, "random"), (1, [100] * 5, 33, 2, 3, 4, "holes"), (90, [50, 0], 64, 2, 5, 32, "random"),     # more
    (400, [100, 7, 0, 250] * 10, 17, 2, 4, 16, "holes"), (500, [0] * 30, 40, 2, 1, 128, "random"), (255, [300, 9] * 30, 20, 1, 2, 2, "holes")])
def test_few_keys_in_one_launch(dfs, D, prefix, lens, T, Hkv, group, page, kind):
    a = make_shared(prefix + T, prefix, lens, T, Hkv, group, D, page, kind)
    for n in sorted({prefix, prefix // 2, 0, min(prefix, 1)}):
        a[7] = i32([n])
        check(dfs, a)
    a[7] = i32([prefix])
    clean = dfs.tree_attention_shared(*a)
    # behind the prefix's end and the sequences' ends, and on pages of nobody, anything may lie
    b = make_shared(prefix + T, prefix, lens, T, Hkv, group, D, page, kind, fill=float("nan"))
    check(dfs, b)
    assert torch.equal(bits(dfs.tree_attention_shared(*a)), bits(clean))
    if prefix > 11:  # seen by all rows but those of unused nodes
        used = ancestors_mask(a[3]).any(dim=2)
        a[5][a[6][11 // page].long(), 0, 11 % page, 5] = float("inf")
        got = dfs.tree_attention_shared(*a)
        assert not torch.isfinite(got[used][:, :group, 5].float()).any() and torch.isfinite(got[used][..., 6:].float()).all()
        assert (got[~used] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix,lens,T,Hkv,group,page,kind", SHARED)
def test_few_keys_in_wide_tables(dfs, D, prefix, lens, T, Hkv, group, page, kind):
    """What goes by the tables' widths goes another way."""
    a = make_shared(prefix + T, prefix, lens, T, Hkv, group, D, page, kind)
    a[6] = wide(a[6], 2000 // page + 1)
    check(dfs, a)
    a[8] = wide(a[8], 9000 // page)
    check(dfs, a)
