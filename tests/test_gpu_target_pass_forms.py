"""Every form that the 8-bit product's rule chooses, on the GPU against its definition in 64 bits.

The rule goes by rows, columns and blocks of k, so each list below names the kernel that its sizes reach:
few rows (one or two tiles of 16), the streaming kernel by its tiles and blocks a wave, and the tiles.
Tolerances are the product's (see test_gpu_target_pass); tests on one value a row and block are exact.
"""
import pytest
import torch

from .test_gpu_target_pass import U, dfs, gen, quantised  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


FEW = [(1, 1000, 272), (16, 5003, 2064), (16, 17001, 5264), (17, 1000, 272), (32, 5003, 1040)]
STREAM = [(5, 16385, 144), (16, 17001, 1040), (16, 17001, 2064), (16, 16389, 3088), (13, 17001, 4112), (16, 20003, 5120),
          (17, 20003, 272), (32, 16391, 1040), (32, 20003, 2064), (29, 17001, 3056)]
WIDE = [(33, 16387, 400), (64, 20003, 2064), (20, 16400, 3200), (48, 16390, 16)]
PAIR = [(33, 130, 272), (150, 300, 1296)]
TALL = [(333, 5003, 272), (640, 6000, 400)]          # bf16; the second one for fp32 too
SMALL = [(512, 5125, 400), (333, 5003, 272)]         # bf16 and fp32; fp32
MID = [(1000, 5003, 272), (1030, 10001, 144)]
BIG = [(4096, 4096, 144), (2049, 7001, 400)]         # bf16; fp32 takes 128 x 128 tiles
ALL = FEW + STREAM + WIDE + PAIR + TALL + SMALL[:1] + MID + BIG
DTYPES = [torch.bfloat16, torch.float32]


def in_64_bits(a, sa, w, sw):
    """(out, the same over magnitudes), a block of k after the other."""
    rows, N = a.shape[0], w.shape[0]
    out = torch.zeros(rows, N, dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(out)
    for g in range(sa.shape[0]):
        x, y = a[:, 128 * g:128 * (g + 1)].double(), w[:, 128 * g:128 * (g + 1)].double()
        f = sa[g].double()[:, None] * sw[:, g].double().repeat_interleave(128)[:N]
        out += (x @ y.t()) * f
        mag += (x.abs() @ y.abs().t()) * f.abs()
    return out, mag


def bound(mag, want, rows, N, K, dtype):
    """The product's tolerance: the 8-bit instruction's loss for a bf16 output in tiles, else fp32 sums, and half a
    step of the output."""
    tiles = rows > 32 or (rows > 16 and N >= 16384 and K > 24 * 128)
    lost = 2.0 ** -10 if dtype == torch.bfloat16 and tiles else (256 + 2 * -(-K // 128) + 12) * U
    return lost * mag + torch.finfo(dtype).eps / 2 * want.abs() + 1e-38


@pytest.mark.parametrize("rows,N,K", STREAM + WIDE + FEW[2:3] + TALL[1:] + SMALL[:1])
def test_accuracy(dfs, rows, N, K):
    g = gen(rows + N + K)
    a, sa = quantised(g, rows, K, 1)
    sa = sa.t().contiguous()
    w, sw = quantised(g, N, K, 128, 0.05)
    want, mag = in_64_bits(a, sa, w, sw)
    for dtype in DTYPES:
        got = dfs.linear_q8(a, sa, w, sw, out_dtype=dtype).double()
        far = ((got - want).abs() / bound(mag, want, rows, N, K, dtype)).max().item()
        assert far <= 1, (dtype, far)


def one_value_a_row(g, rows, N, K):
    """Row r of a has one value, 1, at a k of its own, so that out is w's code there times two powers of two: exact,
    in fp32 and in bf16.  w holds every code but the two NaN."""
    at = torch.randperm(max(rows, K), generator=g, device="cuda")[:rows] % K
    at[-1] = K - 1
    a = torch.zeros(rows, K, device="cuda")
    a[torch.arange(rows, device="cuda"), at] = 1.0
    codes = torch.randint(0, 256, (N, K), generator=g, device="cuda").to(torch.uint8)
    codes = torch.where(codes & 0x7F == 0x7F, codes & 0x80, codes)  # zeros of both signs in their place
    G = -(-K // 128)
    sa = 2.0 ** torch.randint(-6, 7, (G, rows), generator=g, device="cuda").float()
    sw = 2.0 ** torch.randint(-6, 7, (-(-N // 128), G), generator=g, device="cuda").float()
    return a.to(torch.float8_e4m3fn), sa, codes.view(torch.float8_e4m3fn), sw, at


def same(got, want):
    """Equal, NaN for NaN."""
    return bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


@pytest.mark.parametrize("rows,N,K", ALL)
def test_every_code(dfs, rows, N, K):
    a, sa, w, sw, at = one_value_a_row(gen(rows + K), rows, N, K)
    col = torch.arange(N, device="cuda")
    want = w.float()[:, at].t() * sa[at // 128, torch.arange(rows, device="cuda")][:, None] * sw[col // 128][:, at // 128].t()
    for dtype in DTYPES:
        assert same(dfs.linear_q8(a, sa, w, sw, out_dtype=dtype).float(), want), dtype


@pytest.mark.parametrize("rows,N,K", ALL)
def test_infinite_scales(dfs, rows, N, K):
    """An infinite scale of the last block of k, or of a block of columns there: infinite, with the product's sign,
    where the definition is, and NaN only where it is (zero times infinity)."""
    a, sa, w, sw, at = one_value_a_row(gen(rows + K), rows, N, K)
    G = sa.shape[0]
    for side in ("a", "w"):
        sa2, sw2 = sa.clone(), sw.clone()
        if side == "a":
            sa2[G - 1, rows - 1] = float("inf")  # of the row whose value is in that block
        else:
            sw2[-1, G - 1] = float("inf")
        want = in_64_bits(a, sa2, w, sw2)[0]
        for dtype in DTYPES:
            got = dfs.linear_q8(a, sa2, w, sw2, out_dtype=dtype).double()
            assert same(got, want), (side, dtype, int(torch.isnan(got).sum()), int(torch.isnan(want).sum()))


@pytest.mark.parametrize("rows,N,K", ALL)
def test_nan_stays_in_its_row_and_column(dfs, rows, N, K):
    g = gen(N + K)
    a, sa = quantised(g, rows, K, 1)
    sa = sa.t().contiguous()
    w, sw = quantised(g, N, K, 128)
    r, n = rows // 2, N - 1
    a2, w2 = a.clone(), w.clone()
    a2.view(torch.uint8)[r, K - 1] = 0x7F
    w2.view(torch.uint8)[n, K - 16] = 0xFF
    for dtype in DTYPES:
        clean = dfs.linear_q8(a, sa, w, sw, out_dtype=dtype)
        got = dfs.linear_q8(a2, sa, w2, sw, out_dtype=dtype)
        assert torch.isnan(got[r]).all() and torch.isnan(got[:, n]).all()
        got[r], got[:, n] = clean[r], clean[:, n]
        assert torch.equal(got.view(torch.uint8), clean.view(torch.uint8)), dtype


@pytest.mark.parametrize("rows,N,K", [(16, 300, 272), (32, 16400, 272), (33, 16400, 272), (100, 300, 272), (333, 5003, 272),
                                     (512, 5125, 272), (1000, 5003, 272), (2049, 7001, 272)])
def test_large_products_that_cancel(dfs, rows, N, K):
    """448 * 448 and its negative among every eight products.  With an fp32 output, and where rows are few, the sums are
    fp32's; in tiles with a bf16 output a sum is within 2^-10 of the magnitudes, which here is more than what is left."""
    g = gen(K + rows)
    a = torch.randn(rows, K, generator=g, device="cuda")
    w = torch.randn(N, K, generator=g, device="cuda")
    a[:, 1::8], a[:, 6::8] = 448.0, 448.0
    w[:, 1::8], w[:, 6::8] = 448.0, -448.0
    a, w = a.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    G = -(-K // 128)
    sa, sw = torch.ones(G, rows, device="cuda"), torch.ones(-(-N // 128), G, device="cuda")
    want, mag = in_64_bits(a, sa, w, sw)
    for dtype in DTYPES:
        err = (dfs.linear_q8(a, sa, w, sw, out_dtype=dtype).double() - want).abs()
        far = (err / bound(mag, want, rows, N, K, dtype)).max().item()
        print(f"rows {rows} {dtype}: largest error / magnitudes {(err / mag).max().item():.3e}, rms error / rms "
              f"{(err.square().mean() / want.square().mean()).sqrt().item():.3e}", flush=True)
        assert far <= 1, (dtype, far)
