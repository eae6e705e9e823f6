"""Every kernel of the block-scaled product (tests/test_gpu_products.py) on the CPU emulation, one type each
under AddressSanitizer, the smaller ones under ThreadSanitizer too, as tests/test_emu_kernels.py does
for the rest of the library."""

import os

import pytest

from test_emu_inputs import _passed
from test_emu_kernels import ASAN, ROOT, TSAN, _run_selection, build_emu

pytestmark = pytest.mark.skipif(ASAN is None, reason="clang AddressSanitizer runtime not found")

TESTS = "tests/test_gpu_products.py"


def test_products_on_cpu_under_address_sanitizer(tmp_path):
    lib = build_emu.build(out=os.path.join(ROOT, "_build", "emu_products"))
    rc, text = _run_selection(
        tmp_path, lib, ASAN,
        dict(ECHO_EMU_ORDER="5",
             ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0:alloc_dealloc_mismatch=0:"
                          "detect_stack_use_after_return=0:abort_on_error=1"),
        ["-x", TESTS, "-k", "test_forms and bf16 or test_forms_full and fp32 and 128x128 or test_long and 8500 "
                            "or test_long and 33100-fp16"])
    assert rc == 0, text[-6000:]
    assert _passed(text) >= 20, text[-3000:]


@pytest.mark.skipif(TSAN is None, reason="clang ThreadSanitizer runtime not found")
def test_products_on_cpu_under_thread_sanitizer(tmp_path):
    lib = build_emu.build(out=os.path.join(ROOT, "_build", "emu_products_tsan"), sanitizer="thread")
    rc, text = _run_selection(
        tmp_path, lib, TSAN,
        dict(ECHO_EMU_ORDER="6", OPENBLAS_NUM_THREADS="1", OMP_NUM_THREADS="1",
             TSAN_OPTIONS="halt_on_error=0:report_signal_unsafe=0"),
        [TESTS, "-k", "test_forms_full and bf16"])
    assert text.count("WARNING: ThreadSanitizer") == 0, text[text.index("WARNING: ThreadSanitizer"):][:6000]
    assert rc == 0, text[-6000:]
    assert _passed(text) >= 10, text[-3000:]
