"""Rotations at the farthest positions: sine and cosine as they come out, against angles that are exact.

Tolerance (u = 2^-24): the angle is exact but for its remainder's way to fp32, |x| <= pi / 4 with three roundings, 3 u |x|.  That moves the
sine by at most 3 u |x| cos x <= 1.7 u and the cosine by 3 u |x| sin x <= 1.7 u.  The series for a given x: the sine's last step rounds
once, 0.71 u, and has 0.42 u |x| from what it adds; the cosine's 1 u, and 0.64 u from z times its inner sum; left out, 2^-29.
So both are within 3.5 u.  With x1 = 1 and x2 = 0 the turn adds nothing to them.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from .test_gpu_paged_cache import F32, i32
from .test_gpu_target_pass import U, dfs, f64, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
FREQS = [1.0, float(np.float32(0.7310586)), float(np.nextafter(np.float32(1), np.float32(0))), float(np.float32(0.1))]
BOUND = 3.5 * U


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def sine_and_cosine(positions, freqs):
    """[positions, freqs] of either: the angle as a fraction, less whole turns, then in 64 bits."""
    def rest(p, f):
        a = Fraction(int(p)) * Fraction(f)
        return float(a - round(a / (2 * PI)) * 2 * PI)

    a = np.array([[rest(p, f) for f in freqs] for p in positions])
    return np.sin(a), np.cos(a)


def ones(rows, n):
    x = torch.zeros(rows, 1, 2 * n, device="cuda")
    x[..., :n] = 1.0
    return x


def check(y, positions, freqs):
    sine, cosine = sine_and_cosine(positions, freqs)
    n = len(freqs)
    err = np.maximum(np.abs(f64(y)[:, 0, :n] - cosine), np.abs(f64(y)[:, 0, n:] - sine))
    print(f"largest error {err.max() / U:.2f} u", flush=True)
    assert (err <= BOUND).all(), np.unravel_index(err.argmax(), err.shape)


@pytest.mark.parametrize("around", [0, 2 ** 20, 2 ** 27, 2 ** 30, 2 ** 31 - 1, -2 ** 30, -2 ** 31])
def test_far_positions(dfs, around):
    """The last positions of 31 bits as the first ones."""
    rng = np.random.default_rng(abs(around) % 1000)
    pos = np.clip(around + rng.integers(-3000, 3000, 600), -2 ** 31, 2 ** 31 - 1)
    y = dfs.rope(ones(len(pos), 4), None, None, i32(pos.tolist()), torch.tensor(FREQS, device="cuda"))[0]
    check(y, pos, FREQS)


@pytest.mark.parametrize("prefix,length", [(0, 5), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 400), (2 ** 30, 2 ** 31 - 1)])
def test_far_appended_queries(dfs, prefix, length):
    """Positions that are sums: up to 32 bits.  What lies past the table is not written, its query turned all the same."""
    rows = 300
    x = ones(rows, 4)
    pool = torch.zeros(2, 1, 16, 8, device="cuda")
    q, _ = dfs.cache_append(x, x, x, i32([0, rows]), torch.tensor(FREQS, device="cuda"), pool, pool.clone(), i32([[0, 1]]), i32([length]),
                            prefix_len=i32([prefix]))
    check(q, [prefix + length + r for r in range(rows)], FREQS)


def test_frequencies_beyond_any_models(dfs):
    """An angle past 2^53 quarter turns has no digits left, but what comes out is a turn: squares of sine and cosine off by 2 x 3.5 u
    sqrt(2) in all, the turned pair's squares by 2 x 2 u (|x1| + |x2|)^2, at most 8 u of theirs: 18 u."""
    g = gen(3)
    x = randn(g, 64, 3, 8)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (64,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    for f in (1e6, 1e12, 1e20, 3e38):
        y = dfs.rope(x, None, None, pos, torch.full((4,), f, device="cuda"))[0]
        a, b = (t.double()[..., :4].square() + t.double()[..., 4:].square() for t in (x, y))
        assert ((a - b).abs() <= 18 * U * a).all()
    assert x.dtype == F32
