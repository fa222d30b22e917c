"""The host logic of the operators around a paged cache (argument checks, the plans of attention over a shared prefix, the
frequencies' schedules) under AddressSanitizer and UBSan: their tests without a GPU in a child process, on the
host-sanitized build.  CPU only."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _library(build):
    """The host-sanitized library, built unless it is newer than all that it is built from."""
    sources = [os.path.join(d, n) for d in (build.CSRC, os.path.join(ROOT, "include")) for n in os.listdir(d)]
    newest = max(map(os.path.getmtime, [*sources, build.__file__]))
    if os.path.exists(build.SAN_LIB) and os.path.getmtime(build.SAN_LIB) > newest:
        return build.SAN_LIB
    return build.build_host_sanitized()


@pytest.mark.slow
@pytest.mark.parametrize("name", ["test_paged_cache_oracle.py", "test_paged_cache_calls.py"])
def test_under_host_sanitizers(name, tmp_path):
    from draft_selection_position_amd import build

    lib = _library(build)
    env = dict(os.environ)
    rt = build.sanitizer_runtime()
    env["LD_PRELOAD"] = rt + (" " + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = f"detect_leaks=0:log_path={tmp_path / 'asan'}"
    env["UBSAN_OPTIONS"] = f"print_stacktrace=1:log_path={tmp_path / 'ubsan'}"
    env["DFS_LIBRARY"] = lib
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.join(ROOT, "tests", name)],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    reports = sorted(tmp_path.glob("*san*"))
    detail = "".join(f"\n--- {p.name}\n" + p.read_text()[:4000] for p in reports)
    assert r.returncode == 0 and not reports, r.stdout[-4000:] + r.stderr[-4000:] + detail
    assert " passed" in r.stdout and "skipped" not in r.stdout, r.stdout[-2000:]
