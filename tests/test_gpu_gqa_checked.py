"""The grouped-head calls under the checked build (libcsa_checked.so): their shares, output rows, partial states, page
slots and lists are bounds-checked on the device, and a failed check stays in the device error word.  Their tests run in
a child process that loads that library (CSA_LIBRARY), each reading the word; they must pass and leave none recorded."""
import glob
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, torch, pytest
from long_context_sparse_10_b200 import _lib
assert _lib.LIB_PATH.endswith("libcsa_checked.so"), _lib.LIB_PATH
rc = pytest.main(["-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_gqa.py",
                  "-k", "paged_chunks or packed_prompts or weight or evict or append or rows_without or many or outside"])
lib = _lib.load()
st = lib.csa_check_device_error(torch.cuda.current_stream().cuda_stream)
print("device error status", st, lib.csa_last_error())
sys.exit(int(rc) if rc else (0 if st == 0 else 7))
"""


def test_every_unit_has_checks():
    from long_context_sparse_10_b200 import build
    paths = [p for p in sorted(glob.glob(os.path.join(build.CSRC, "gqa*.cu"))) if "_global__" in open(p).read()]
    assert len(paths) == 3
    for path in paths:
        assert re.search(r"CSA_INBOUNDS\(", open(path).read()), path


@pytest.mark.gpu
def test_grouped_heads_and_no_bounds_failure_under_the_checked_build():
    from long_context_sparse_10_b200 import build
    path = build.LIB_CHECKED
    if not os.path.exists(path):
        build.build(checked=True)
    env = dict(os.environ, CSA_LIBRARY=path)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
