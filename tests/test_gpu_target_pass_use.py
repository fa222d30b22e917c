"""The verification pass's operators as they are used: one after the other, on other streams, captured and
replayed, with offsets past 32 bits, and refusals by the binding."""
import numpy as np
import pytest
import torch

from oracle import target_pass as tp

from .test_gpu_target_pass import (cache, check_attention, check_linear, check_norm, dfs, f64, gen, make, quantised,  # noqa: F401
                                   randn, trees)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def linear_tol(a, sa, w, sw, out):
    want, mag = tp.linear_q8(f64(a), f64(sa), f64(w), f64(sw))
    # bf16 out: 2^-10 of the magnitudes for the 8-bit matrix instruction (see the product's tests), half a step
    return want, (2.0 ** -10 * mag if out.dtype == torch.bfloat16 else 400 * 2.0 ** -24 * mag) + 2.0 ** -8 * np.abs(want) + 1e-30


class Layer:
    """Weights of one small layer and a head, quantised once."""

    def __init__(self, g, d, Hq, Hkv, D, V):
        self.d, self.Hq, self.Hkv, self.D, self.V = d, Hq, Hkv, D, V
        self.norm = (1 + 0.1 * randn(g, d)).bfloat16()
        self.qkv = quantised(g, (Hq + 2 * Hkv) * D, d, 128, d ** -0.5)
        self.o = quantised(g, d, Hq * D, 128, (Hq * D) ** -0.5)
        self.head = quantised(g, V, d, 128, d ** -0.5)
        self.ones = torch.ones(Hq * D, dtype=torch.bfloat16, device="cuda")


def verification_pass(dfs, layer, x, res, parents, pools, table, lens, trace=None):
    """One layer over the nodes' hidden states, then the head: (logits fp32, k_new, v_new)."""
    B, T, _ = x.shape
    q8, sc, res = dfs.norm_q8(x, layer.norm, res)
    qkv = dfs.linear_q8(q8, sc, *layer.qkv)
    Hq, Hkv, D = layer.Hq, layer.Hkv, layer.D
    q, k, v = (t.reshape(B, T, -1, D).contiguous() for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
    att = dfs.tree_attention(q, k, v, parents, *pools, table, lens)
    a8, asc = dfs.norm_q8(att.reshape(B, T, -1), layer.ones)
    o = dfs.linear_q8(a8, asc, *layer.o)
    h8, hsc, res2 = dfs.norm_q8(o, layer.norm, res)
    logits = dfs.linear_q8(h8, hsc, *layer.head, out_dtype=torch.float32)
    if trace is not None:
        trace.update(q8=q8, sc=sc, qkv=qkv, q=q, k=k, v=v, att=att, a8=a8, asc=asc, o=o, h8=h8, hsc=hsc, res=res)
    return logits, k, v


def test_a_pass_over_drafted_blocks(dfs):
    """Norm, projections, attention, head, verification of the drafted path, commit, and the next pass: each step
    against the oracle on what it was given, and the committed cache against the nodes' own keys."""
    g = gen(21)
    B, T, d, Hq, Hkv, D, V = 5, 6, 512, 8, 2, 64, 4000
    layer = Layer(g, d, Hq, Hkv, D, V)
    lens = [0, 17, 64, 100, 5]
    kp, vp, table, ln = cache(g, lens, Hkv, D, 16, spare=2 * T)
    x, r, par = randn(g, B, T, d, dtype=torch.bfloat16), randn(g, B, T, d, dtype=torch.bfloat16), trees(g, B, T, "chain")
    tr = {}
    logits, k, v = verification_pass(dfs, layer, x, r, par, (kp, vp), table, ln, tr)
    check_norm((tr["q8"], tr["sc"], tr["res"]), x, layer.norm, r, 1e-6, False)
    flat = lambda t: t.reshape(B * T, -1)  # noqa: E731
    for a, s, (w, sw), out in ((tr["q8"], tr["sc"], layer.qkv, tr["qkv"]), (tr["a8"], tr["asc"], layer.o, tr["o"]),
                               (tr["h8"], tr["hsc"], layer.head, logits)):
        want, tol = linear_tol(flat(a), s, w, sw, out)
        assert (np.abs(f64(flat(out)) - want) <= tol).all()
    check_attention(dfs, tr["q"], k, v, par, kp, vp, table, ln, got=tr["att"])

    # the drafted path against these logits: what a verifier keeps of it goes into the cache
    cand, val = dfs.topk(logits)
    path = cand[:, 1:, 0].contiguous()
    qd = torch.zeros(B, T - 1, 16, device="cuda")
    qd[:, :, 0] = 1.0
    accepted, token = dfs.verify(logits, path, cand[:, 1:].contiguous(), qd, temperature=1.0, seed=3)
    counts = accepted + 1
    k2, v2 = kp.clone(), vp.clone()
    new = dfs.cache_commit(k, v, None, counts, k2, v2, table, ln)
    assert torch.equal(new, ln + counts)
    wk, wv, _ = tp.cache_commit(f64(k), f64(v), None, counts.tolist(), f64(kp), f64(vp), table.cpu().numpy(), lens)
    np.testing.assert_array_equal(f64(k2), wk)
    np.testing.assert_array_equal(f64(v2), wv)
    # the next pass reads them
    nx = randn(g, B, 1, d, dtype=torch.bfloat16)
    tr2 = {}
    verification_pass(dfs, layer, nx, nx, trees(g, B, 1, "chain"), (k2, v2), table, new, tr2)
    check_attention(dfs, tr2["q"], tr2["k"], tr2["v"], trees(g, B, 1, "chain"), k2, v2, table, new, got=tr2["att"])


def test_committed_nodes_equal_seen_ones(dfs):
    """The last node of a path sees the same keys whether the nodes before it are in the tree or in the cache."""
    q, k, v, par, kp, vp, table, ln = make(31, [33, 0, 200], 9, 2, 3, 128, 16)
    g = gen(31)
    B, T = 3, 9
    kp, vp, table, ln = cache(g, [33, 0, 200], 2, 128, 16, spare=T)
    whole = dfs.tree_attention(q, k, v, par, kp, vp, table, ln)
    counts = torch.full((B,), T - 1, dtype=torch.int32, device="cuda")
    new = dfs.cache_commit(k, v, None, counts, kp, vp, table, ln)
    one = lambda t: t[:, -1:].contiguous()  # noqa: E731
    got = dfs.tree_attention(one(q), one(k), one(v), trees(g, B, 1, "chain"), kp, vp, table, new)
    check_attention(dfs, one(q), one(k), one(v), trees(g, B, 1, "chain"), kp, vp, table, new, got=got)
    # each is within 2^-8 of the weighted |v| (weights) and 2^-8 of itself (output) of the same sum, both at most
    # the largest |v|: twice two half steps of that, and one more for the fp32 terms
    most = max(vp.abs().max().item(), v.abs().max().item())
    assert (got - whole[:, -1:]).abs().max() <= 5 * 2.0 ** -8 * most


def test_the_same_call_gives_the_same_bits(dfs):
    a = make(41, [700, 3, 4000, 64], 17, 2, 4, 128, 64, "random")
    first = dfs.tree_attention(*a)
    g = gen(42)
    x, s = quantised(g, 40, 2064, 1)
    s = s.t().contiguous()
    w, sw = quantised(g, 20000, 2064, 128)
    y = dfs.linear_q8(x, s, w, sw)
    for _ in range(5):
        assert torch.equal(dfs.tree_attention(*a).view(torch.int16), first.view(torch.int16))
        assert torch.equal(dfs.linear_q8(x, s, w, sw).view(torch.int16), y.view(torch.int16))


def test_two_streams_at_once(dfs):
    calls = [make(50 + i, [900, 10 + i], 5, 2, 4, 64, 16) for i in range(2)]
    want = [dfs.tree_attention(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(dfs.tree_attention(*calls[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for t in got[i]:
            assert torch.equal(t.view(torch.int16), want[i].view(torch.int16))


def test_captured_and_replayed(dfs):
    """Two graphs of a pass each, replayed with eager work and synchronisation between, on changed inputs."""
    g = gen(61)
    B, T, d, Hq, Hkv, D, V = 3, 4, 512, 8, 2, 64, 3000
    layer = Layer(g, d, Hq, Hkv, D, V)
    kp, vp, table, ln = cache(g, [30, 0, 77], Hkv, D, 16, spare=T)
    par = trees(g, B, T, "random")
    counts = torch.tensor([2, 4, 0], dtype=torch.int32, device="cuda")
    inputs = [randn(g, B, T, d, dtype=torch.bfloat16) for _ in range(4)]

    def work(x):
        logits, k, v = verification_pass(dfs, layer, x, x, par, (kp, vp), table, ln)
        return [logits, dfs.cache_commit(k, v, None, counts, kp, vp, table, ln), k]

    static = [inputs[0].clone(), inputs[1].clone()]
    work(static[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in static:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work(x))
        graphs.append(graph)
    for turn in range(6):
        for i in range(2):
            static[i].copy_(inputs[(turn + i) % 4])
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            mine = [t.clone() for t in outs[i]]
            pools = kp.clone(), vp.clone()
            eager = work(static[i])  # the same commit again
            for a, b in zip(mine, eager):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (turn, i)
            assert torch.equal(pools[0], kp) and torch.equal(pools[1], vp)


def test_a_node_that_is_not_finite_in_q(dfs):
    a = make(71, [50, 130], 20, 2, 2, 64, 16, "random")
    want = dfs.tree_attention(*a)
    a[0][0, 7, 1] = float("nan")
    got = dfs.tree_attention(*a)
    assert torch.isnan(got[0, 7, 1].float()).all()
    got[0, 7, 1] = want[0, 7, 1]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_a_pool_past_32_bits(dfs):
    g = gen(81)
    Hkv, page, D = 8, 64, 128
    n = 40000  # 5.2 GB a pool
    kp, vp = (torch.empty((n, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = [130, 70]
    table = torch.tensor([[n - 1, 39000, n - 3, n - 7], [n - 2, 38999, 0, 0]], dtype=torch.int32, device="cuda")
    for p in table.flatten().tolist():
        kp[p], vp[p] = randn(g, Hkv, page, D, dtype=torch.bfloat16), randn(g, Hkv, page, D, dtype=torch.bfloat16)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    B, T = 2, 3
    q, k, v = randn(g, B, T, Hkv, D, dtype=torch.bfloat16), randn(g, B, T, Hkv, D, dtype=torch.bfloat16), randn(g, B, T, Hkv, D, dtype=torch.bfloat16)
    par = trees(g, B, T, "chain")
    new = dfs.cache_commit(k, v, None, torch.tensor([2, 3], dtype=torch.int32, device="cuda"), kp, vp, table, ln)
    assert torch.equal(kp[n - 3, :, 130 % 64 + 1], k[0, 1]) and torch.equal(vp[38999, :, 70 % 64 + 2], v[1, 2])
    out = dfs.tree_attention(q, k, v, par, kp, vp, table, new)
    used = sorted(set(table.flatten().tolist()))
    small = torch.tensor([[used.index(p) for p in row] for row in table.tolist()], dtype=torch.int32, device="cuda")
    check_attention(dfs, q, k, v, par, kp[used], vp[used], small, new, got=out)


def test_a_product_past_32_bits(dfs):
    g = gen(82)
    rows, N, K = 4100, 530000, 128  # 2.2e9 outputs
    a, sa = quantised(g, rows, K, 1)
    w, sw = quantised(g, N, K, 128)
    sa = sa.t().contiguous()
    out = dfs.linear_q8(a, sa, w, sw)
    for r in (0, 4099):
        for n in (0, N - 300):
            want, tol = linear_tol(a[r:r + 1], sa[:, r:r + 1], w[n // 128 * 128:][:300], sw[n // 128:][:3], out)
            got = f64(out[r:r + 1, n // 128 * 128:][:, :300])
            assert (np.abs(got - want) <= tol).all()


def test_a_norm_past_32_bits(dfs):
    g = gen(83)
    rows, d = 270000, 8192  # 2.2e9 values
    x = torch.randn((rows, d), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    q, s = dfs.norm_q8(x, w)
    pick = [0, 1, 262143, 262144, rows - 1]
    check_norm((q[pick], s[:, pick]), x[pick], w, None, 1e-6, False)


# ---------------------------------------------------------------- the binding's refusals


def test_binding_refuses(dfs):
    g = gen(91)
    x, w = randn(g, 4, 256, dtype=torch.bfloat16), randn(g, 256, dtype=torch.bfloat16)
    for bad, kind in (((x.float(), w), ValueError), ((x.half(), w.half()), ValueError), ((x.t(), w), ValueError),
                      ((x, w[:128]), ValueError), ((x.cpu(), w.cpu()), ValueError), ((x, w.cpu()), ValueError),
                      ((None, w), TypeError), ((x, None), TypeError)):
        with pytest.raises(kind):
            dfs.norm_q8(*bad)
    for kw in (dict(residual=x[:2]), dict(residual=x.float()), dict(total_out=x), dict(residual=x, total_out=x[:2])):
        with pytest.raises(ValueError):
            dfs.norm_q8(x, w, **kw)
    with pytest.raises(dfs.DfsError):
        dfs.norm_q8(x[:0], w)
    with pytest.raises(dfs.DfsError):
        dfs.norm_q8(x[:, :24].contiguous(), w[:24].contiguous())
    a, sa = quantised(g, 4, 256, 1)
    sa = sa.t().contiguous()
    b, sb = quantised(g, 200, 256, 128)
    for bad in ((a, sa.t(), b, sb), (a, sa, b, sb[:1]), (a.float(), sa, b, sb), (a, sa, b[:, :128].contiguous(), sb),
                (a, sa.double(), b, sb), (a, sa.cpu(), b, sb)):
        with pytest.raises(ValueError):
            dfs.linear_q8(*bad)
    with pytest.raises(ValueError):
        dfs.linear_q8(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        dfs.linear_q8(a, sa, b, sb, out=torch.empty(4, 200, device="cuda"))
    at = make(92, [20, 3], 3, 2, 2, 64, 16)
    for i, bad in ((0, at[0].float()), (0, at[0][:, :2].contiguous()), (1, at[1].float()), (1, at[1][:1]), (2, None), (3, at[3].long()),
                   (3, at[3][:1]), (4, at[4][:, :1].contiguous()), (5, at[5][1:]), (6, at[6][:1]), (7, at[7].cpu()), (7, at[7].long())):
        with pytest.raises((ValueError, TypeError)):
            dfs.tree_attention(*at[:i], bad, *at[i + 1:])
    with pytest.raises(ValueError):
        dfs.tree_attention(*make(92, [2000, 3], 3, 2, 2, 64, 16), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dfs.DfsError):
        dfs.tree_attention(*at, scale=0.0)
    with pytest.raises(dfs.DfsError):
        dfs.tree_attention(*at, out=at[0])
    counts = torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dfs.cache_commit(at[1], at[2], None, counts[:1], *at[4:])
    with pytest.raises(ValueError):
        dfs.cache_commit(at[1], at[2], counts, counts, *at[4:])
    with pytest.raises(dfs.DfsError):
        dfs.cache_commit(at[1], at[2], None, counts, *at[4:], out_lens=at[7])


def test_explicit_workspace(dfs):
    a = make(93, [500], 4, 2, 2, 64, 16)
    n = dfs.tree_attention_workspace_bytes(1, 4, 4, 2, 64, 16, a[4].shape[0], a[6].shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(dfs.tree_attention(*a, workspace=ws), dfs.tree_attention(*a))
