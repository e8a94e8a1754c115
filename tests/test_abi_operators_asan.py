"""The operators' host code under AddressSanitizer, on the CPU, as
test_abi_asan.py has the block's: the argument checks, the launch shapes and the
workspace arithmetic run in a child process on the host-only sanitizer build."""

import os
import subprocess
import sys

import pytest

from test_abi_asan import CHILD, ROOT


@pytest.mark.parametrize("name", ["test_abi_operators.py", "test_abi_operators_sizes.py"])
def test_operators_host_code_under_address_sanitizer(name):
    from group_limited_routing_amd import build
    rt = build.asan_runtime()
    if rt is None:
        pytest.skip("no AddressSanitizer runtime next to hipcc's clang")
    tests = os.path.join(ROOT, "tests")
    lib = build.ASAN_LIB_PATH
    newest = max(os.path.getmtime(os.path.join(build.CSRC, f)) for f in os.listdir(build.CSRC))
    if not os.path.exists(lib) or os.path.getmtime(lib) < newest:
        lib = build.build(asan=True)
    env = dict(os.environ, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:exitcode=99")
    code = CHILD.format(root=ROOT, tests=tests, lib=lib, abi=os.path.join(tests, name))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=600, cwd=ROOT)
    assert "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-2000:])
    assert "passed" in r.stdout
