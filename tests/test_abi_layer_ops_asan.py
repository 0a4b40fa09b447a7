"""The refusals of the int8 products, SwiGLU, the sum over slots and the layer for
a few tokens under AddressSanitizer and UndefinedBehaviorSanitizer (host code;
see test_abi_asan.py)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.slow
def test_refusals_under_asan_ubsan(tmp_path):
    from bit_rank_post_amd import build as B
    try:
        B.hipcc()
        rt = B.asan_runtime()
    except (RuntimeError, OSError, subprocess.CalledProcessError) as e:
        pytest.skip(f"sanitizer toolchain unavailable: {e}")
    log = str(tmp_path / "sanitizer")
    env = dict(os.environ, LD_PRELOAD=rt, TILEQ_LIB_PATH=B.build_asan(),
               ASAN_OPTIONS=f"detect_leaks=0:abort_on_error=0:log_path={log}",
               UBSAN_OPTIONS=f"halt_on_error=1:print_stacktrace=1:log_path={log}")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_layer_ops.py"), "-k", "not on_the_host and not torch and not offered"],
                       cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=600)
    reports = [os.path.join(tmp_path, f) for f in os.listdir(tmp_path) if f.startswith("sanitizer")]
    text = "".join(open(f).read()[:4000] for f in reports)
    assert r.returncode == 0 and not reports, (r.stdout.decode(errors="replace")[-3000:] + text)
    assert b"passed" in r.stdout
