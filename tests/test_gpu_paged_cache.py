"""The operators around a paged cache on the GPU against the fp64 oracle (oracle/paged_cache.py).

Tolerances, from fp32 arithmetic (u = 2^-24 per rounding) and each output's own rounding (half a step):
  rotation   the quarter turns q = position freq 2 / pi in 64 bits, two roundings: their angle is off by at most
             pi / 2 |q| 2^-52.  What is left of it, |x| <= pi / 4, has three roundings to fp32: 3 u |x| <= 2.4 u;
             the series one more in its last step, half of one before it, and what they leave out, 2^-29: 1.6 u.
             The amplitude and its product: 2 u.  So sine and cosine are within 6 u A.  x1 c - x2 s: one rounding of a
             product, one of the sum: (6 + 2) u A (|x1| + |x2|) in all.  The output: half a step.  Values that are
             copied keep their bits.
  attention  as tree attention without a prefix: weights rounded to bf16, 2^-8 of sum w |v|; a score's error
             (D + 4) u sum |q k| scale and the exponential's argument (2^7 u) change a weight by that much relative,
             numerator and denominator: twice.  Sums over n keys 2 n u; joins of pieces, 64 of them at most here, two
             roundings each: 128 u.  The output: 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import paged_cache as pc

from .test_gpu_target_pass import U, cache, dfs, f64, gen, randn, trees  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- positions


@pytest.mark.parametrize("B,T,kind", [(1, 1, "chain"), (3, 17, "chain"), (5, 64, "random"), (70, 63, "holes"), (4, 33, "holes"),
                                      (1000, 2, "random")])
def test_positions(dfs, B, T, kind):
    g = gen(B + T)
    par = trees(g, B, T, kind)
    lens = torch.randint(0, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = -5
    for prefix in (None, 0, 12345):
        got = dfs.tree_positions(par, lens, None if prefix is None else i32([prefix]))
        assert np.array_equal(got.cpu().numpy(), pc.tree_positions(par.tolist(), lens.tolist(), prefix or 0))


def test_positions_of_odd_parents_and_lengths(dfs):
    big = 2 ** 31 - 1
    par = i32([[0, 0, 1, -1], [big, -big, 1, 2], [-1, 0, 1, 2], [-1, -1, 5, 2]])
    lens = i32([3, 4, big, 1 << 30])
    for prefix in (-7, 0, big):
        got = dfs.tree_positions(par, lens, i32([prefix]))
        assert np.array_equal(got.cpu().numpy(), pc.tree_positions(par.tolist(), lens.tolist(), prefix))


# ---------------------------------------------------------------- rotation


def rotation_tol(want, mag, positions, freqs, dtype):
    quarters = np.abs(np.outer(positions, freqs)).max(initial=0.0) * 2 / np.pi
    half = torch.finfo(dtype).eps / 2
    return mag * (8 * U + quarters * 2.0 ** -52 * np.pi / 2) + half * np.abs(want) + 1e-37


def check_rotated(got, x, positions, freqs, layout, amplitude):
    """got, x [rows, heads, D]"""
    f = f64(freqs)
    want, mag = pc.rotate(f64(x), positions, f, layout, float(np.float32(amplitude)))
    err, tol = np.abs(f64(got) - want), rotation_tol(want, mag, positions, f, x.dtype)
    assert (err <= tol).all(), (np.unravel_index((err - tol).argmax(), err.shape), (err / tol).max())
    n = 2 * len(f)
    as_is = torch.int16 if x.dtype == BF16 else torch.int32
    assert torch.equal(got[..., n:].contiguous().view(as_is), x[..., n:].contiguous().view(as_is))


def frequencies(rot, factor=1.0):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / factor).float().cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rows,Hq,Hkv,D,rot", [
    (1, 1, 1, 8, 2), (1, 32, 8, 128, 128), (5, 4, 2, 64, 64), (3, 7, 3, 80, 20), (4, 3, 1, 96, 24), (2, 5, 5, 96, 96),
    (7, 2, 1, 256, 64), (3, 1, 1, 1024, 1024), (2, 3, 2, 520, 130), (3, 2, 1, 1024, 6), (2, 40, 9, 72, 36), (1, 3, 1, 16, 14),
    (67, 9, 2, 64, 32)])
def test_rope(dfs, dtype, layout, rows, Hq, Hkv, D, rot):
    g = gen(rows + D + rot)
    qkv = randn(g, rows, Hq + 2 * Hkv, D, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, device="cuda", dtype=torch.int32)
    f = frequencies(rot)
    oq, ok, ov = dfs.rope(q, k, v, pos, f, layout=layout, amplitude=1.25)
    assert oq.is_contiguous() and ok.is_contiguous() and torch.equal(ov, v)
    check_rotated(oq, q, pos.tolist(), f, layout, 1.25)
    check_rotated(ok, k, pos.tolist(), f, layout, 1.25)
    # the same from dense inputs, each alone, and in place
    dq, dk = q.contiguous(), k.contiguous()
    assert torch.equal(dfs.rope(dq, None, None, pos, f, layout=layout, amplitude=1.25)[0], oq)
    assert torch.equal(dfs.rope(None, dk, v, pos, f, layout=layout, amplitude=1.25)[1], ok)
    got = dfs.rope(dq, dk, None, pos, f, layout=layout, amplitude=1.25, out=(dq, dk, None))
    assert got[0] is dq and torch.equal(dq, oq) and torch.equal(dk, ok) and got[2] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rope_far_and_negative_positions(dfs, dtype):
    g = gen(5)
    pos = [0, 1, -1, -1000003, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31]
    x = randn(g, len(pos), 2, 64, dtype=dtype)
    f = frequencies(64)
    check_rotated(dfs.rope(x, None, None, i32(pos), f)[0], x, pos, f, "half", 1.0)
    one = torch.ones(32, device="cuda")
    check_rotated(dfs.rope(x, None, None, i32(pos), one)[0], x, pos, one, "half", 1.0)


def test_rope_every_quadrant(dfs):
    """Angles around the borders of the quarter turns, where quadrant and remainder change together."""
    pos = list(range(-40, 41))
    for f0 in (np.pi / 2, np.pi / 4, 3 * np.pi / 4, 1.0, 0.0):
        f = torch.full((4,), float(np.float32(f0)), device="cuda")
        x = randn(gen(6), len(pos), 1, 8)
        check_rotated(dfs.rope(x, None, None, i32(pos), f)[0], x, pos, f, "half", 1.0)


def test_rope_many_rows(dfs):
    """More rows than take a wave for every pass over their heads: the same bits as row by row."""
    g = gen(7)
    rows = 20011
    qkv = randn(g, rows, 48, 64, dtype=BF16)
    pos = torch.randint(0, 100000, (rows,), generator=g, device="cuda", dtype=torch.int32)
    f = frequencies(64)
    q, k, v = dfs.rope(qkv[:, :32], qkv[:, 32:40], qkv[:, 40:], pos, f)
    pick = [0, 1, 2, 63, 64, 10000, rows - 1]
    for r in pick:
        one = dfs.rope(qkv[r:r + 1, :32], qkv[r:r + 1, 32:40], qkv[r:r + 1, 40:], pos[r:r + 1], f)
        assert torch.equal(one[0][0], q[r]) and torch.equal(one[1][0], k[r]) and torch.equal(one[2][0], v[r])
    check_rotated(q[pick], qkv[pick, :32], pos[pick].tolist(), f, "half", 1.0)
    assert torch.equal(v, qkv[:, 40:])


def test_rope_what_is_not_finite_stays_in_its_pair(dfs):
    x = randn(gen(8), 2, 2, 16, dtype=BF16)
    f, pos = frequencies(8), i32([3, 4])
    want = dfs.rope(x, None, None, pos, f)[0]
    x[0, 1, 2] = float("inf")
    x[1, 0, 9] = float("nan")  # behind what is turned
    got = dfs.rope(x, None, None, pos, f)[0]
    bad = ~torch.isfinite(got.float())
    assert bad.nonzero().tolist() == [[0, 1, 2], [0, 1, 6], [1, 0, 9]]
    assert torch.equal(got[~bad], want[~bad])


def test_rope_leading_dimensions(dfs):
    g = gen(9)
    qkv = randn(g, 3, 5, 8, 64, dtype=BF16)
    pos = torch.randint(0, 5000, (3, 5), generator=g, device="cuda", dtype=torch.int32)
    f = frequencies(64)
    q, k, _ = dfs.rope(qkv[:, :, :6], qkv[:, :, 6:], None, pos, f)
    flat = dfs.rope(qkv.view(15, 8, 64)[:, :6], qkv.view(15, 8, 64)[:, 6:], None, pos.view(15), f)
    assert q.shape == (3, 5, 6, 64) and torch.equal(q.view(15, 6, 64), flat[0]) and torch.equal(k.view(15, 2, 64), flat[1])
    with pytest.raises(ValueError, match="evenly"):
        dfs.rope(qkv[:, :4], None, None, pos[:, :4].contiguous(), f)


# ---------------------------------------------------------------- append


def run_append(dfs, starts, lens, rows, Hq, Hkv, D, rot, page, layout, dtype, seed, prefix=None, with_q=True, spare=0):
    g = gen(seed)
    B = len(lens)
    room = [max(0, n) + max(0, starts[b + 1] - starts[b]) for b, n in enumerate(lens)]
    kp, vp, table, _ = cache(g, room, Hkv, D, page, dtype=dtype)
    if spare:  # some sequences' last pages missing
        table[:, -spare:] = -1
    qkv = randn(g, rows, Hq + 2 * Hkv, D, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    f = frequencies(rot) if rot else None
    k0, v0, ln = kp.clone(), vp.clone(), i32(lens)
    mark = torch.full((rows, Hq, D), 7.0, dtype=dtype, device="cuda")
    oq, new = dfs.cache_append(q if with_q else None, k, v, i32(starts), f, kp, vp, table, ln, layout=layout,
                               prefix_len=None if prefix is None else i32([prefix]), q_out=mark if with_q else None)
    assert new.tolist() == [max(0, n) + starts[b + 1] - starts[b] for b, n in enumerate(lens)]
    slots = pc.append_slots(starts, rows, table.cpu().numpy(), lens, kp.shape[0], page, prefix or 0)
    mine = [r for r, s in enumerate(slots) if s is not None]
    pos = [slots[r][0] for r in mine]
    if with_q:
        if mine:
            check_rotated(oq[mine], q[mine], pos, f if rot else torch.empty(0), layout, 1.0)
        rest = [r for r in range(rows) if slots[r] is None]
        assert (oq[rest] == 7.0).all()  # rows that are no tokens
    put = [r for r in mine if slots[r][1] is not None]
    if put:
        at = torch.tensor([slots[r][1:] for r in put], device="cuda")
        check_rotated(kp[at[:, 0], :, at[:, 1]], k[put], [slots[r][0] for r in put], f if rot else torch.empty(0), layout, 1.0)
        assert torch.equal(vp[at[:, 0], :, at[:, 1]], v[put])
        k0[at[:, 0], :, at[:, 1]] = kp[at[:, 0], :, at[:, 1]]
        v0[at[:, 0], :, at[:, 1]] = vp[at[:, 0], :, at[:, 1]]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)  # and nothing else


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("starts,lens,rows,Hq,Hkv,D,rot,page,layout,prefix", [
    ([0, 1], [0], 1, 1, 1, 8, 8, 1, "half", None),
    ([0, 17], [4001], 17, 32, 8, 128, 128, 16, "half", 0),
    ([0, 0, 5, 5, 6], [3, 0, 9, 15], 6, 4, 2, 64, 32, 16, "interleaved", 1000),  # sequences without tokens
    ([2, 4, 9], [7, 0], 12, 3, 1, 80, 20, 4, "half", None),                      # rows in front and behind that are none
    ([0, 3, 3], [0, 5], 3, 2, 2, 96, 48, 2, "interleaved", 3),
    ([0, 0], [5], 3, 2, 1, 64, 64, 16, "half", None),                             # no tokens at all
    ([0, 40], [100], 40, 2, 1, 256, 256, 32, "half", 70000),
])
def test_append(dfs, dtype, starts, lens, rows, Hq, Hkv, D, rot, page, layout, prefix):
    run_append(dfs, starts, lens, rows, Hq, Hkv, D, rot, page, layout, dtype, rows + D, prefix)
    run_append(dfs, starts, lens, rows, Hq, Hkv, D, rot, page, layout, dtype, rows + D, prefix, with_q=False)
    run_append(dfs, starts, lens, rows, Hq, Hkv, D, 0, page, layout, dtype, rows + D, prefix)


@pytest.mark.parametrize("B", [63, 64, 65, 200, 4097, 5000])
def test_append_many_sequences(dfs, B):
    """Either side of the batches whose sequences' ends a wave reads at once."""
    rng = np.random.default_rng(B)
    counts = rng.integers(0, 3, B) * (rng.random(B) < 0.5)
    starts = np.concatenate([[0], np.cumsum(counts)]).tolist()
    run_append(dfs, starts, rng.integers(0, 20, B).tolist(), starts[-1] + 3, 2, 1, 16, 16, 4, "half", BF16, B)


def test_append_past_the_table(dfs):
    run_append(dfs, [0, 30, 41], [5, 60], 41, 2, 1, 64, 64, 8, "half", BF16, 3, spare=3)


def test_append_lengths_and_pages_out_of_range(dfs):
    run_append(dfs, [0, 4, 9], [-7, 3], 9, 1, 1, 64, 64, 4, "half", BF16, 4)
    g = gen(11)
    kp, vp, table, _ = cache(g, [20], 1, 64, 4)
    table[0, 1], table[0, 2], table[0, 3] = kp.shape[0], -1, 2 ** 31 - 1
    x = randn(g, 20, 3, 64, dtype=BF16)
    k0 = kp.clone()
    pages = table[0].tolist()
    _, new = dfs.cache_append(None, x[:, :1], x[:, 1:2], i32([0, 20]), None, kp, vp, table, i32([0]))
    assert new.tolist() == [20]
    for t in (0, 4):
        assert torch.equal(kp[pages[t], 0], x[4 * t:4 * t + 4, 0])
        k0[pages[t]] = kp[pages[t]]
    assert torch.equal(kp, k0)
    # a length so large that no table has it
    _, new = dfs.cache_append(None, x[:, :1], x[:, 1:2], i32([0, 20]), None, kp, vp, table, i32([2 ** 31 - 3]))
    assert new.tolist() == [2 ** 31 - 1] and torch.equal(kp, k0)


def test_append_starts_that_are_not_in_order(dfs):
    """Outside the contract, but nothing may be written outside the tokens' own pages."""
    g = gen(12)
    B, rows = 200, 50
    kp, vp, table, ln = cache(g, [8] * B, 1, 64, 4)
    table.clamp_(min=0)
    x = randn(g, rows, 2, 64, dtype=BF16)
    for kind in range(4):
        starts = torch.randint(-5, 100, (B + 1,), generator=g, device="cuda", dtype=torch.int32)
        if kind == 1:
            starts = starts.sort(descending=True).values
        if kind == 2:
            starts[:] = -2 ** 31
        if kind == 3:
            starts[::2], starts[1::2] = 2 ** 31 - 1, -2 ** 31
        dfs.cache_append(None, x[:, :1], x[:, 1:], starts, None, kp, vp, table, ln)
        torch.cuda.synchronize()


# ---------------------------------------------------------------- attention over a shared prefix


def make_shared(seed, prefix, lens, T, Hkv, group, D, page, kind="chain", fill=None, qstd=1.5):
    g = gen(seed)
    B = len(lens)
    kp, vp, table, ln = cache(g, lens + [prefix], Hkv, D, page, fill=fill)
    width = max(1, -(-max(lens) // page)) + 1
    return [randn(g, B, T, Hkv * group, D).mul(qstd).bfloat16(), randn(g, B, T, Hkv, D, dtype=BF16),
            randn(g, B, T, Hkv, D, dtype=BF16), trees(g, B, T, kind), kp, vp, table[B].contiguous(), i32([prefix]),
            table[:B, :width].contiguous(), ln[:B].contiguous()]


def check_shared(dfs, q, kn, vn, par, kp, vp, ptab, plen, table, lens, scale=None, got=None):
    out = dfs.tree_attention_shared(q, kn, vn, par, kp, vp, ptab, plen, table, lens, scale) if got is None else got
    D = q.shape[-1]
    sc = D ** -0.5 if scale is None else scale
    want, mag, dots, keys = pc.tree_attention_shared(f64(q), f64(kn), f64(vn), par.tolist(), f64(kp), f64(vp),
                                                     ptab.cpu().numpy(), int(plen), table.cpu().numpy(), lens.tolist(), sc)
    tol = mag * (2.0 ** -8 + 2 * ((D + 4) * U * dots + 2.0 ** 7 * U) + (2 * keys + 128) * U)[..., None] + 2.0 ** -8 * np.abs(want) + 1e-30
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), (np.unravel_index((err / tol).argmax(), err.shape), (err / tol).max())
    print(f"largest error / bound {(err / tol).max():.3f}", flush=True)


SHARED = [
    (0, [0], 1, 1, 1, 1, "chain"),                 # nothing but the node itself
    (1, [0], 1, 1, 1, 1, "chain"),
    (0, [5, 40], 3, 2, 2, 16, "random"),           # no prefix
    (200, [0, 0, 0], 2, 2, 4, 16, "chain"),        # nothing but the prefix
    (31, [1], 1, 2, 1, 16, "chain"),
    (32, [3, 0], 4, 1, 3, 32, "random"),
    (33, [70], 1, 3, 8, 1, "chain"),
    (127, [130, 2, 64], 5, 1, 2, 64, "holes"),
    (129, [0, 9, 33, 100], 4, 2, 4, 16, "random"),  # 64 rows in all
    (64, [10] * 5, 17, 1, 1, 16, "chain"),         # 85
    (300, [77, 5], 33, 2, 2, 128, "holes"),        # 132
    (1000, [0, 200], 64, 1, 3, 256, "random"),     # 384
    (517, [0, 1, 2, 3, 60] * 10, 7, 2, 1, 16, "holes"),  # 350
    (77, [20] * 70, 3, 1, 2, 8, "random"),         # more sequences than a wave has lanes
    (4100, [17, 300, 0], 2, 2, 4, 64, "chain"),
    (130, [(7 * b) % 90 for b in range(40)] + [900, 0, 1500], 3, 2, 2, 64, "random"),  # cut ones, many in one part
    (50, [600] + [(11 * b) % 70 for b in range(90)], 17, 1, 4, 16, "chain"),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix,lens,T,Hkv,group,page,kind", SHARED)
def test_shared(dfs, D, prefix, lens, T, Hkv, group, page, kind):
    check_shared(dfs, *make_shared(prefix + T, prefix, lens, T, Hkv, group, D, page, kind))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_shared_what_no_sequence_owns_is_not_read(dfs, D, fill):
    """Pages end inside tiles: whatever lies behind a sequence's last key, or the prefix's, reaches nobody."""
    for prefix, lens, T, page in ((37, [5, 0], 3, 16), (200, [130, 1], 40, 64), (0, [9, 9], 2, 8), (700, [0] * 40, 8, 128)):
        check_shared(dfs, *make_shared(prefix, prefix, lens, T, 1, 2, D, page, "random", fill=fill))


def test_shared_unused_nodes(dfs):
    """A tree of unused nodes only: zeros, whatever its queries hold; the others as they were."""
    a = make_shared(21, 300, [40, 7, 0], 12, 2, 2, 64, 16)
    a[3][1] = -2
    a[0][1] = float("nan")
    out = dfs.tree_attention_shared(*a)
    assert (out[1] == 0).all()
    a[0][1] = 0
    check_shared(dfs, *a, got=out)


def test_shared_scores_far_apart(dfs):
    """Weights of the prefix, or of the sequence's own keys, that vanish beside the other's."""
    for big in ("prefix", "own"):
        a = make_shared(22, 150, [90, 30], 4, 1, 2, 128, 16, qstd=1.0)
        q, kp, ptab, table = a[0], a[4], a[6], a[8]
        q.fill_(1.0)
        pages = ptab[:10].long() if big == "prefix" else table[:, :6].clamp(min=0).unique().long()
        kp[pages] = kp[pages] * 0.1 + 12.0
        check_shared(dfs, *a)


def test_shared_large_scores(dfs):
    a = make_shared(23, 500, [100, 3], 9, 2, 2, 64, 16, "random", qstd=40.0)
    check_shared(dfs, *a)
    check_shared(dfs, *a, scale=1e-30)


def test_shared_infinite_scores(dfs):
    """A key whose scores are all -inf weighs nothing; rows that see nothing else are zero."""
    a = make_shared(24, 20, [0, 0], 1, 1, 1, 64, 4)
    a[0].fill_(1.0)
    a[1].fill_(-float("inf"))  # the nodes' own keys
    out = dfs.tree_attention_shared(*a)
    a[3][:] = -1
    kp, vp, ptab = a[4], a[5], a[6]
    pos = torch.arange(20, device="cuda")
    k, v = (p[ptab[pos // 4].long(), 0, pos % 4].double() for p in (kp, vp))
    w = torch.softmax(a[0][0, 0].double() @ k.t().contiguous() / 8, dim=1)
    assert (out[:, 0].double() - (w @ v)).abs().max() <= 3 * 2.0 ** -8 * v.abs().max()
    a[7] = i32([0])
    assert (dfs.tree_attention_shared(*a) == 0).all()


def test_shared_lengths_out_of_range(dfs):
    """A prefix's length beyond its table, or below zero; entries of the tables that point nowhere."""
    a = make_shared(25, 64, [20, 5], 3, 1, 2, 64, 16)
    a[6] = a[6][:4].contiguous()
    want = dfs.tree_attention_shared(*a)
    a[7] = i32([2 ** 31 - 1])
    assert torch.equal(dfs.tree_attention_shared(*a), want)
    none = a[:7] + [i32([0])] + a[8:]
    a[7] = i32([-3])
    assert torch.equal(dfs.tree_attention_shared(*a), dfs.tree_attention_shared(*none))
    a[7] = i32([64])
    n = a[4].shape[0]
    a[6] = i32([2 ** 31 - 1, -5, n, 0])
    clamped = a[:6] + [i32([n - 1, 0, n - 1, 0])] + a[7:]
    assert torch.equal(dfs.tree_attention_shared(*a), dfs.tree_attention_shared(*clamped))


def test_shared_equals_unshared(dfs):
    """The same keys with the prefix's pages at the head of every sequence's own table."""
    page = 16
    for D, T, group, kind in ((64, 9, 2, "random"), (128, 1, 4, "chain"), (128, 17, 4, "holes")):
        a = make_shared(26, 32 * page, [40, 0, 333, 16], T, 2, group, D, page, kind)
        q, kn, vn, par, kp, vp, ptab, plen, table, lens = a
        B = len(lens)
        both = torch.cat([ptab[None, :32].expand(B, -1), table], dim=1).contiguous()
        want = dfs.tree_attention(q, kn, vn, par, kp, vp, both, lens + 32 * page)
        got = dfs.tree_attention_shared(*a)
        # both are within 2^-8 (weights) of the weighted |v| and 2^-8 of themselves, and a little more
        most = max(vp.float().abs().max().item(), vn.float().abs().max().item())
        assert (got.float() - want.float()).abs().max() <= 5 * 2.0 ** -8 * most
        check_shared(dfs, *a, got=got)
