"""The decode kernel's plan, computed on the host for a sweep of shapes: rings of an even number of
stages (a stage that passes from one MMA issuer to the other may be read before its copy has landed),
at least two of them, within the shared memory of a CTA."""
from __future__ import annotations

import subprocess

from int8_quantized_02_b200 import build as build_mod

MAIN = r"""
#include <cstdio>
#include "kernels.h"
namespace llmint8 { void note_launches(int) {} }
int main() {
    const long caps[] = {0, 1, 16, 64, 100, 256}, ns[] = {16, 128, 1024, 4096, 11008, 16384, 20000, 38100, 49152, 100000};
    long n = 0, bad = 0, rings = 0;
    for (long M = 1; M <= llmint8::kDecodeMaxM; ++M)
        for (long cap : caps)
            for (long N : ns)
                for (long K = 16; K <= llmint8::kDecodeMaxK; K += 16) {
                    const llmint8::DecodePlan p = llmint8::decode_plan(M, N, K, cap, 148);
                    const bool ok = p.stages >= 2 && p.stages % 2 == 0 && p.smem <= 232448 &&
                                    (p.resident ? p.nistage == p.nst : p.nistage % 2 == 0);
                    ++n, rings += !p.resident, bad += !ok;
                }
    std::printf("%ld %ld %ld\n", n, rings, bad);
}
"""


def test_rings_are_even(tmp_path):
    main, exe = tmp_path / "main.cu", tmp_path / "plan"
    main.write_text(MAIN)
    arch = build_mod.NVCC_FLAGS[:2]
    subprocess.run([build_mod._nvcc(), *arch, "-std=c++17", f"-I{build_mod.INCLUDE}", f"-I{build_mod.CSRC}",
                    "-o", str(exe), str(main), f"{build_mod.CSRC}/decode.cu"], check=True, timeout=600)
    n, rings, bad = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                                            timeout=600).stdout.split())
    assert n == 16 * 6 * 10 * 1024 and rings > 0 and bad == 0
