"""The operators in front of the scores (page maps, FP8 in blocks of 128, head norms with rotation,
the indexer's inputs) on the CPU emulation: their GPU parity tests under AddressSanitizer and under
ThreadSanitizer, as tests/test_emu_kernels.py does for the rest of the library (its docstring says
what this catches)."""

import os
import re

import pytest

from test_emu_kernels import ASAN, ROOT, TSAN, _run_selection, build_emu

pytestmark = pytest.mark.skipif(ASAN is None, reason="clang AddressSanitizer runtime not found")

SELECTION = ["tests/test_gpu_pages.py", "tests/test_gpu_blockfp8.py", "tests/test_gpu_heads.py", "tests/test_gpu_inputs.py",
             "-k", "not full"]


def _passed(text):
    m = re.search(r"(\d+) passed", text)
    return int(m.group(1)) if m else 0


def test_input_operators_on_cpu_under_address_sanitizer(tmp_path):
    lib = build_emu.build(out=os.path.join(ROOT, "_build", "emu_inputs"))
    rc, text = _run_selection(
        tmp_path, lib, ASAN,
        dict(ECHO_EMU_ORDER="3",
             ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0:alloc_dealloc_mismatch=0:"
                          "detect_stack_use_after_return=0:abort_on_error=1"),
        ["-x", *SELECTION])
    assert rc == 0, text[-6000:]
    assert _passed(text) >= 100, text[-3000:]


@pytest.mark.skipif(TSAN is None, reason="clang ThreadSanitizer runtime not found")
def test_input_operators_on_cpu_under_thread_sanitizer(tmp_path):
    lib = build_emu.build(out=os.path.join(ROOT, "_build", "emu_inputs_tsan"), sanitizer="thread")
    rc, text = _run_selection(
        tmp_path, lib, TSAN,
        dict(ECHO_EMU_ORDER="4", OPENBLAS_NUM_THREADS="1", OMP_NUM_THREADS="1",
             TSAN_OPTIONS="halt_on_error=0:report_signal_unsafe=0"),
        SELECTION)
    assert text.count("WARNING: ThreadSanitizer") == 0, text[text.index("WARNING: ThreadSanitizer"):][:6000]
    assert rc == 0, text[-6000:]
    assert _passed(text) >= 100, text[-3000:]
