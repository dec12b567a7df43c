"""The MXFP4 products under the debug build (libllmint8_debug.so): their device-side checks of tiles,
stages and stores hold on the shapes of the tests, whose status must be LLMINT8_OK there."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from int8_quantized_02_b200 import build as build_mod

pytestmark = pytest.mark.gpu


def test_products_pass_under_the_debug_build():
    build_mod.build(debug=True)
    env = dict(os.environ, LLMINT8_DEBUG="1")
    run = subprocess.run(
        [sys.executable, "-c",
         "import sys, pytest; from int8_quantized_02_b200 import llmint8 as L; assert L.build_flags() & 1; "
         "sys.exit(pytest.main(['tests/test_mxfp4_gpu.py', '-m', 'gpu', '-q', '-x', '-p', 'no:cacheprovider', "
         "'-k', '(test_linear and not dtype1) or streams or run_of']))"],
        cwd=build_mod.ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert run.returncode == 0, run.stdout[-4000:] + run.stderr[-2000:]
    assert " passed" in run.stdout
