"""Which entries of the page tables attention over a short shared prefix reads (CPU: the kernel's own function, on the
host)."""
import os
import subprocess

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "pins", "page_entry.cpp")


@pytest.fixture(scope="module")
def page_entry(tmp_path_factory):
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available to build it")
    exe = str(tmp_path_factory.mktemp("page_entry") / "page_entry")
    subprocess.run([hipcc, "--offload-arch=gfx950", "-O1", SOURCE, "-o", exe], check=True, capture_output=True)
    return exe


def test_entries_within_the_lengths_alone(page_entry):
    """Nothing behind the prefix's length, nor behind a sequence's: with neither, no entry of either table."""
    cases = [(f, n, s) for f in (0, 1, 2, 31, 32, 33, 64, 100) for n in (0, 1, 5, 32, 70) for s in (0, 1, 4, 7)]
    text = "".join(f"{f} {n} {s}\n" for f, n, s in cases)
    lines = subprocess.run([page_entry], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.splitlines()
    assert len(lines) == len(cases)
    for (f, n, s), line in zip(cases, lines):
        keys = [min(k, f + n - 1) for k in range(f + n + 64)]
        want = [f"P{k >> s}" if 0 <= k < f else f"T{(k - f) >> s}" if n else "L" for k in keys]
        assert line.split() == want, (f, n, s)
