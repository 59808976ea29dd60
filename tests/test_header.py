"""The header for C and C++ programs: it compiles without a warning, and every
constant is a value that its type has."""
import os
import subprocess

import pytest

import mxfp4_block_scaled_fp4q_amd as fq
from mxfp4_block_scaled_fp4q_amd import build

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
CONSTANTS = dict(FP4Q_F32=0, FP4Q_BF16=1, FP4Q_SILU=fq.SILU, FP4Q_GELU=fq.GELU, FP4Q_LAYER_NORM=fq.LAYER_NORM,
                 FP4Q_RMS_NORM=fq.RMS_NORM, FP4Q_NO_NORM=fq.NO_NORM, FP4Q_NORM_L2=fq.NORM_L2,
                 FP4Q_NORM_MAX=fq.NORM_MAX)


@pytest.mark.parametrize("language", ["c", "c++"])
def test_constants_are_values_of_their_types(tmp_path, language):
    check = "_Static_assert" if language == "c" else "static_assert"
    source = tmp_path / "use.c"
    source.write_text('#include "libfp4q.h"\n' + "".join(
        f'{check}({name} == {value}, "{name}");\n' for name, value in CONSTANTS.items())
        + "fp4q_norm_t none(void) { return FP4Q_NO_NORM; }\n")
    clang = os.path.join(os.path.dirname(os.path.dirname(build._hipcc())), "llvm", "bin", "clang")
    std = "c11" if language == "c" else "c++17"
    for compiler in (clang, "gcc"):
        run = subprocess.run([compiler, "-x", language, f"-std={std}", "-Wall", "-Wextra", "-Werror", "-fsyntax-only",
                              "-I", INCLUDE, str(source)], capture_output=True, text=True)
        assert run.returncode == 0, f"{compiler} {language}: {run.stderr[:1500]}"
