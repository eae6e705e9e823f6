"""The package without parts that it does not need (no GPU, nothing compiled)."""

import os
import subprocess
import sys

import pytest

from dsa_indexer_top_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="library not built")
def test_binding_and_library_load_without_torch():
    """Callers that bring their own device memory need no torch: only calls that take tensors do."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from dsa_indexer_top_amd import binding as B\n"
            "assert 'gfx950' in B.version() and B.page_workspace_bytes(4, 16) > 0\n"
            "assert B.lib().echo_topk is not None\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
