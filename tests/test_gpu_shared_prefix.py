"""Every way that attention over a shared prefix takes, against a dense computation in 64 bits on the GPU: the prefix's
own kernel (many rows, a long table), one launch for both, own keys by single waves, own keys in a launch of their own.

Which way is taken goes by the sizes and the tables' widths, not by the lengths: wide tables with few keys behind them
reach all of them at sizes that the dense computation has room for.  Tolerances as in test_gpu_paged_cache.py.
"""
import pytest
import torch

from .test_gpu_paged_cache import BF16, i32, make_shared
from .test_gpu_target_pass import U, dfs, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ancestors_mask(parents):
    """[B, T, T]: whether node t sees node u."""
    B, T = parents.shape
    node = torch.arange(T, device=parents.device)
    p = parents.long()
    used = (p >= -1) & (p < node)
    up = (p[:, :, None] == node) & used[:, :, None] & used[:, None, :]
    sees = torch.eye(T, dtype=torch.float64, device=p.device) * used[:, :, None]
    step = torch.eye(T, dtype=torch.float64, device=p.device) + up.double()
    reach = torch.matrix_power(step, max(T, 1)) if T > 1 else step
    return ((reach > 0) & used[:, :, None] & used[:, None, :]) | (sees > 0)


def dense64(q, kn, vn, par, kp, vp, ptab, plen, table, lens, scale):
    """(out, sum of weights |v|, largest sum |q k| scale of a row, keys of a row), by kv head."""
    B, T, Hq, D = q.shape
    Hkv, page = kp.shape[1:3]
    g, P = Hq // Hkv, int(plen)
    lens = lens.clamp(0, table.shape[1] * page).long()
    S = int(lens.max())
    pos, own = torch.arange(P, device=q.device), torch.arange(S, device=q.device)
    there = own < lens[:, None]
    pages = torch.where(there, table.long()[:, own // page], 0).clamp(0, kp.shape[0] - 1)
    tree = ancestors_mask(par)
    out, mag = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    dots, keys = (torch.zeros(B, T, Hq, dtype=torch.float64, device=q.device) for _ in range(2))
    alive = tree.any(dim=2)
    near = torch.cat([there[:, None, :].expand(B, T, S), tree], dim=2)  # [B, T, S + T]
    for h in range(Hkv):
        x = q[:, :, h * g:(h + 1) * g].double()  # [B, T, g, D]
        flat, rows = x.reshape(B * T * g, D), x.reshape(B, T * g, D)
        far = [p[ptab.long()[pos // page], h, pos % page].double() for p in (kp, vp)]  # [P, D]
        by = [torch.cat([torch.where(there[..., None], p[pages, h, own % page].double(), 0.0), n[:, :, h].double()], dim=1)
              for p, n in ((kp, kn), (vp, vn))]  # [B, S + T, D]
        see = near.repeat_interleave(g, dim=1)
        part = lambda a, b: torch.cat([(flat_(a) @ far[0].abs().t().contiguous() if b else flat_(a) @ far[0].t().contiguous()).view(B, T * g, P),  # noqa: E731
                                       a @ (by[0].abs() if b else by[0]).transpose(1, 2).contiguous()], dim=2)
        flat_ = lambda a: a.reshape(B * T * g, D)  # noqa: E731
        s = part(rows, False) * scale
        seen = torch.cat([torch.ones(B, T * g, P, dtype=torch.bool, device=q.device), see], dim=2)
        seen &= alive.repeat_interleave(g, dim=1)[:, :, None]
        s = s.masked_fill(~seen, -float("inf"))
        top = s.amax(dim=2, keepdim=True)
        w = torch.exp(s - torch.where(top == -float("inf"), 0.0, top))
        total = w.sum(dim=2, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
        mix = lambda f, b: ((w[..., :P].reshape(B * T * g, P) @ f).view(B, T * g, D) + w[..., P:] @ b).view(B, T, g, D)  # noqa: E731
        out[:, :, h * g:(h + 1) * g], mag[:, :, h * g:(h + 1) * g] = mix(far[1], by[1]), mix(far[1].abs(), by[1].abs())
        d = part(rows.abs(), True).masked_fill(~seen, 0.0).amax(dim=2) * scale
        dots[:, :, h * g:(h + 1) * g], keys[:, :, h * g:(h + 1) * g] = d.view(B, T, g), seen.sum(dim=2).double().view(B, T, g)
    return out, mag, dots, keys


def check(dfs, a, scale=None, got=None):
    out = dfs.tree_attention_shared(*a, scale=scale) if got is None else got
    D = a[0].shape[-1]
    want, mag, dots, keys = dense64(*a, D ** -0.5 if scale is None else scale)
    tol = mag * (2.0 ** -8 + 2 * ((D + 4) * U * dots + 2.0 ** 7 * U) + (2 * keys + 128) * U)[..., None] + 2.0 ** -8 * want.abs() + 1e-30
    err = (out.double() - want).abs()
    worst = (err / tol).max().item()
    assert (err <= tol).all(), ((err / tol).argmax().item(), worst)
    print(f"largest error / bound {worst:.3f}", flush=True)


def wide(t, width):
    """A table with entries behind its own that point nowhere."""
    pad = torch.full((*t.shape[:-1], max(0, width - t.shape[-1])), -(1 << 30), dtype=torch.int32, device=t.device)
    return torch.cat([t, pad], dim=-1).contiguous()


def large(a):
    """The same call with a prefix table wide enough for the prefix's own kernel."""
    B, T, Hq, D = a[0].shape
    Hkv, page = a[4].shape[1:3]
    need = -(-3 * 2 ** 32 // (B * T * (Hq // Hkv) * Hkv * D))
    assert B * T * (Hq // Hkv) > 384 and need <= 2 ** 30
    a[6] = wide(a[6], -(-need // page) + 1)
    return a


LARGE = [  # prefix, own lengths, T, kv heads, group, page, tree
    (0, [3] * 100, 4, 1, 1, 16, "chain"),             # no prefix at all
    (1, [0] * 100, 1, 2, 4, 1, "chain"),              # a single key; pages smaller than a load's rows
    (31, [5] * 50, 9, 1, 1, 2, "random"),
    (32, [0] * 97, 4, 3, 1, 4, "holes"),
    (33, [17] * 30, 1, 8, 13, 8, "chain"),            # 390 rows
    (63, [1] * 6, 64, 2, 2, 16, "random"),            # 768 rows: three whole row tiles
    (64, [9] * 200, 1, 1, 2, 64, "chain"),
    (65, [0, 70] * 20, 11, 1, 1, 32, "holes"),
    (127, [12] * 33, 4, 2, 3, 64, "random"),
    (128, [0] * 65, 2, 1, 3, 128, "chain"),
    (129, [30] * 40, 17, 4, 1, 16, "random"),
    (1000, [40] * 64, 2, 5, 4, 16, "chain"),          # 51 workgroups a head
    (2047, [3] * 100, 4, 2, 1, 64, "holes"),
    (4100, [100, 0, 7, 300] * 8, 17, 1, 1, 256, "random"),
    (9001, [20] * 16, 7, 2, 4, 64, "chain"),
    (700, [2] * 40, 3, 33, 4, 16, "random"),          # seven workgroups a head, two row tiles
    (650, [2] * 80, 7, 64, 2, 16, "chain"),           # four workgroups a head, five row tiles: whole ones and a rest
    (300, [0] * 200, 2, 128, 3, 16, "chain"),         # two a head
    (90, [0] * 130, 3, 300, 1, 8, "chain"),           # one a head, heads past the card's workgroups
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix,lens,T,Hkv,group,page,kind", LARGE)
def test_large(dfs, D, prefix, lens, T, Hkv, group, page, kind):
    check(dfs, large(make_shared(prefix + T, prefix, lens, T, Hkv, group, D, page, kind)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 128])
def test_large_every_end(dfs, D, page):
    """Prefixes that end at every place of a step's 32 or 64 keys, and ranges of one step and more."""
    a = large(make_shared(7 + page, 700, [3] * 130, 1, 1, 3, D, page))
    for n in (*range(1, 68), 95, 96, 97, 190, 191, 192, 193, 255, 257, 319, 383, 385, 511, 513, 640, 641, 700):
        a[7] = i32([n])
        check(dfs, a)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_large_what_no_sequence_owns_is_not_read(dfs, D, fill):
    for prefix, page in ((37, 16), (100, 1), (200, 64), (1001, 128)):
        check(dfs, large(make_shared(prefix, prefix, [5, 0, 130] * 45, 3, 1, 1, D, page, "random", fill=fill)))


@pytest.mark.parametrize("D", [64, 128])
def test_large_maxima_that_rise(dfs, D):
    """Scores that rise along the prefix, so that sums are rescaled again and again, or fall, so that never; large ones; keys
    whose scores are -inf, all of a step's and some."""
    a = large(make_shared(31, 1500, [9] * 100, 4, 1, 1, D, 64, qstd=1.0))
    q, kp, ptab = a[0], a[4], a[6]
    q.copy_(q.abs() + 0.5)
    pos = torch.arange(1500, device="cuda")
    at = (ptab[pos // 64].long(), slice(None), pos % 64)
    was = kp[at].clone()
    for ramp in (torch.linspace(-2, 4, 1500), torch.linspace(4, -2, 1500), torch.linspace(-2, 4, 1500)[torch.randperm(1500)]):
        kp[at] = (was.float() * 0.3 + ramp.cuda()[:, None, None]).bfloat16()
        check(dfs, a)
    check(dfs, a, scale=3.0)
    kp[at] = was
    kp[ptab[:3].long()] = -float("inf")  # q > 0: scores of -inf
    kp[ptab[5].long(), :, 3:60] = -float("inf")
    want, mag, dots, keys = dense64(*[x.clone() if i == 4 else x for i, x in enumerate(a)], D ** -0.5)
    out = dfs.tree_attention_shared(*a)
    finite = torch.where(torch.isfinite(kp.float()), kp.float(), 0.0).bfloat16()
    dots = dense64(*a[:4], finite, *a[5:], D ** -0.5)[2]  # of the keys that count
    tol = mag * (2.0 ** -8 + 2 * ((D + 4) * U * dots + 2.0 ** 7 * U) + (2 * keys + 128) * U)[..., None] + 2.0 ** -8 * want.abs() + 1e-30
    assert ((out.double() - want).abs() <= tol).all()
    # all of the prefix, its end inside a step too: nothing but the rest counts
    kp[ptab[:24].long()] = -float("inf")
    for n in (1500, 100, 1):
        a[7] = i32([n])
        none = a[:7] + [i32([0])] + a[8:]
        got, rest = dfs.tree_attention_shared(*a).float(), dense64(*none, D ** -0.5)
        assert ((got - rest[0]).abs() <= rest[1] * 2.0 ** -7 + 2.0 ** -8 * rest[0].abs() + 1e-30).all()


@pytest.mark.parametrize("D", [64, 128])
def test_large_not_finite_where_it_is_seen(dfs, D):
    """A NaN in a query stays in its row; one in the prefix's V reaches every row that is not a node's that is unused."""
    a = large(make_shared(32, 300, [9] * 100, 5, 1, 1, D, 16, "holes"))
    want = dfs.tree_attention_shared(*a)
    used = ancestors_mask(a[3]).any(dim=2)
    b, t = used.nonzero()[7].tolist()
    a[0][b, t] = float("nan")
    got = dfs.tree_attention_shared(*a)
    assert torch.isnan(got[b, t].float()).all()
    got[b, t] = want[b, t]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    a[0][b, t] = 0.5
    a[5][a[6][3].long(), 0, 2, 11] = float("nan")
    got = dfs.tree_attention_shared(*a)
    assert torch.isnan(got[used][..., 11].float()).all() and torch.isfinite(got[used][..., :11].float()).all()
    assert (got[~used] == 0).all()


def test_large_lengths_and_pages_out_of_range(dfs):
    a = large(make_shared(33, 96, [4] * 100, 4, 1, 1, 64, 16))
    a[7] = i32([-5])
    assert torch.equal(dfs.tree_attention_shared(*a), dfs.tree_attention_shared(*a[:7], i32([0]), *a[8:]))
    n = a[4].shape[0]
    a[7] = i32([96])
    a[6][:6] = i32([2 ** 31 - 1, -5, n, 0, 1, -1])
    b = list(a)
    b[6] = a[6].clone()
    b[6][:6] = i32([n - 1, 0, n - 1, 0, 1, 0])
    assert torch.equal(dfs.tree_attention_shared(*a), dfs.tree_attention_shared(*b))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix,lens,T,Hkv,group,page,own_width,kind", [
    (100, [(7 * b) % 90 for b in range(600)], 1, 2, 4, 16, 0, "chain"),         # a wave each: 1200 of them
    (0, [0] * 1024, 2, 1, 1, 16, 0, "random"),
    (1, [1] * 300, 8, 4, 4, 16, 0, "holes"),                                    # 32 rows each
    (333, [2000, 1, 0] * 350, 3, 1, 2, 1, 0, "random"),                         # longer own keys than a wave takes
    (333, [70, 1, 0] * 350, 3, 1, 2, 16, 200, "random"),                        # too wide a table for that
    (500, [600, 0, 33], 2, 2, 4, 16, 600, "random"),                            # own keys in a launch of their own
    (500, [900, 5], 20, 1, 2, 16, 600, "holes"),
    (64, [100] * 4, 64, 2, 1, 16, 600, "chain"),
    (700, [9, 0, 300, 64], 17, 2, 4, 64, 0, "random"),                          # one launch, 272 rows
    (700, [9] * 10, 9, 3, 1, 64, 0, "chain"),                                   # 90 rows
    (40, [3000, 0], 64, 1, 7, 64, 0, "holes"),                                  # 896 rows, few products
])
def test_other_ways(dfs, D, prefix, lens, T, Hkv, group, page, own_width, kind):
    a = make_shared(prefix + T + len(lens), prefix, lens, T, Hkv, group, D, page, kind)
    a[8] = wide(a[8], own_width)
    check(dfs, a)


@pytest.mark.parametrize("D", [64, 128])
def test_large_with_every_kind_of_own_keys(dfs, D):
    """The prefix's own kernel beside own keys by single waves, cut over workgroups, and long ones."""
    for lens, T, Hkv, group, width in (([(5 * b) % 60 for b in range(600)], 1, 2, 4, 0), ([900, 0, 30, 2000, 5] * 2, 17, 1, 4, 0),
                                       ([9000, 3, 0, 70], 25, 1, 4, 0), ([3] * 40, 12, 1, 1, 4000)):
        a = large(make_shared(41, 450, lens, T, Hkv, group, D, 16, "random"))
        a[8] = wide(a[8], width)
        check(dfs, a)
