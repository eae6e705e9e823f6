"""The package's loading and building without parts that it does not need (no GPU, nothing compiled)."""

import os
import subprocess
import sys

import pytest

from dsa_indexer_top_amd import binding, build

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


def test_library_is_linked_where_the_tensor_calls_do_not_build(monkeypatch, tmp_path):
    """The native module of the tensor calls needs torch's headers and a host compiler; without them
    the C library is built all the same, and the failure is raised after it."""
    linked = []

    def link(cmd, **kw):
        linked.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def no_module():
        raise RuntimeError("no torch headers")

    monkeypatch.setattr(build, "OUT", str(tmp_path / "libecho.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(build, "_tensor_calls", no_module)
    monkeypatch.setattr(build.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="no torch headers"):
        build.build()
    assert len(linked) == 1 and os.path.exists(build.OUT)
